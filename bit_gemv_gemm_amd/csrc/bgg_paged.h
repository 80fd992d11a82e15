// What the attention kernels over a paged cache share: lane moves, the
// element types of their matrix products, the registers of a tile of the
// cache, and the pass over infinite values.
#pragma once
#include <hip/hip_runtime.h>

#include <cfloat>

#include "bgg_cache.h"
#include "bgg_lowp.h"

namespace bgg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kTokens = 32;  // tokens of a tile: one wave's step
constexpr int kHeads = 16;   // query heads of a workgroup (columns of the products)

// A sequence of a batch whose groups share prefixes: the parts of its group's,
// of key head kh's head i, are rows row + (chunk * kv_heads + kh) * rows + i of
// the prefix parts.
struct SharedSeq {
  int32_t chunks, rows, row;
};
// An Item without its head block.
struct OwnItem {
  int32_t b, chunk, chunks, part, lo, n, tile, tile_end;
};

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  float* lse;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lengths;
  int64_t window;
  uint32_t* counters;
  float* parts;
  float scale;
  int max_tokens, pages, batch, q_heads, kv_heads, group, head_blocks, page_shift;
  int target_items;
  // sequences that share a prefix (bgg_shared_attention)
  const int32_t *group_starts, *shared_pages;
  int groups, prefix_target;
  int own_target, own_chunks;  // items of own tokens (as target_items); chunks of a sequence at most
  int32_t* own_count;  // [1]: entries of own_items
  OwnItem* own_items;
  SharedSeq* seqs;     // [batch]
  float* prefix_parts;
};

struct Item {
  int b, head_block;  // head_block = key head * head_blocks + block of 16 of its query heads
  int chunk, chunks;
  int part;            // of a sequence with several chunks: this one among all such
  int lo, n;           // visible tokens
  int tile, tile_end;  // this chunk's tiles (token / 32)
};

__device__ __forceinline__ void visible(const AttnParams& p, int b, int& lo, int& n) {
  const int len = p.lengths[b];
  n = len < 0 ? 0 : len < p.max_tokens ? len : p.max_tokens;
  lo = p.window > 0 && n > p.window ? n - (int)p.window : 0;
}
// A sequence of up to kOneChunk tiles stays whole: the join costs more than
// the chunks gain (one sequence of 500 tokens, 8 x 128 f16: chunks of 4, 8,
// 16 tiles 10.3, 11.2, 9.2 us).  A longer one is joined in any case; a wave's
// tile costs about 1.2 us of latency and a part 0.15 us of the join, so up to
// 128 tiles a chunk has at least about sqrt(tiles / 2) of them (chunks of 4,
// 8, 16 tiles: 1024 tokens 10.0, 10.8, 12.9 us; 2048 11.7, 11.3, 13.3; 8192
// 17.6, 17.4, 15.8).  The floor stays at 16 for longer sequences, whose even
// share is more than that with eight head blocks; with one or two it is not,
// and longer chunks are not measured there (1 x 65536 tokens: 16 heads on one
// key head, 128 parts, 36 us; 8 on two 26; 1 x 262144: 68 and 54, their bytes
// 22 and 44).
constexpr int kOneChunk = 16;
__device__ __forceinline__ int chunks_of(int tiles, int size) {
  if (tiles <= kOneChunk) return 1;
  size = max(size, tiles <= 32 ? 4 : tiles <= 128 ? 8 : 16);
  return (tiles + size - 1) / size;
}

__device__ __forceinline__ int both_counts(int chunks) {
  return chunks | (chunks > 1 ? chunks << 16 : 0);
}

// Floats of a part: rows of D accumulators, then each row's maximum and sum.
__host__ __device__ constexpr int64_t part_floats(int64_t rows, int64_t D) {
  return (rows * (D + 2) + 3) / 4 * 4;
}
// Chunks of a sequence at most (the items of one sequence and head block,
// about target_items of which there are kMaxItems at most).
constexpr int kMaxItems = 256, kMaxChunks = kMaxItems + 1;
// (a workgroup of one wave holds the weights of fewer parts)
__host__ __device__ constexpr int most_chunks(int waves) { return waves == 1 ? 64 : kMaxChunks; }

// ---------------------------------------------------------------------------
// lane moves
// ---------------------------------------------------------------------------
// Sum over the lanes up to and including this one.
__device__ __forceinline__ int scan_add(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2, 3
  return v;
}
template <int MOVE, int ROWS>
__device__ __forceinline__ float add_from(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), MOVE, ROWS, 0xF, false));
}
// Sum over all lanes, in every lane.
__device__ __forceinline__ float wave_add(float v) {
  v = add_from<0x111, 0xF>(v);
  v = add_from<0x112, 0xF>(v);
  v = add_from<0x114, 0xF>(v);
  v = add_from<0x118, 0xF>(v);
  v = add_from<0x142, 0xA>(v);
  v = add_from<0x143, 0xC>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// Maximum and sum over the four lanes that hold one column (l, l ^ 16,
// l ^ 32, l ^ 48).
__device__ __forceinline__ float column_max(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ int tiles_of(int lo, int n) {
  return n > lo ? (n - 1) / kTokens - lo / kTokens + 1 : 0;
}

// ---------------------------------------------------------------------------
// Element types of the products: q.k in the type of q, the probabilities and
// values in the cache's 16-bit type (fp16 for E4M3, whose values fp16 holds).
// ---------------------------------------------------------------------------
template <class T>
struct Mma;
template <>
struct Mma<F16> {
  using op = f16x8;
  // a probability is at most 2^(7 + kSlack) = 2^15, inside fp16, and fp16's
  // subnormals begin at 2^-21 of the maximum
  static constexpr float lift = 7.0f;
  static __device__ __forceinline__ f32x4 mul(op a, op b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ op round(const float (&v)[8]) {
    op r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (_Float16)v[i];
    return r;
  }
  static __device__ __forceinline__ op split(const float (&v)[8], float (&rest)[8]) {
    op r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[i] = (_Float16)v[i];
      rest[i] = v[i] - (float)r[i];
    }
    return r;
  }
  // four e4m3 bytes -> four values
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t* out) {
    out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
  }
};
template <>
struct Mma<BF16> {
  using op = bf16x8;
  // a probability is at most 1, so that the largest bfloat16 values stay
  // inside fp32
  static constexpr float lift = -8.0f;
  static __device__ __forceinline__ f32x4 mul(op a, op b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ op round(const float (&v)[8]) {
    op r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
    return r;
  }
  static __device__ __forceinline__ op split(const float (&v)[8], float (&rest)[8]) {
    op r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r[i] = (__bf16)v[i];
      rest[i] = v[i] - (float)r[i];
    }
    return r;
  }
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t* out) {
    out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
  }
};
template <class T, class C>
struct ValueType {
  using type = C;
};
template <class T>
struct ValueType<T, E4M3> {
  using type = F16;
};

template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* out) {
  if constexpr (BYTES == 16) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
    out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    out[0] = v.x, out[1] = v.y;
  } else if constexpr (BYTES == 4) {
    out[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    static_assert(BYTES == 2, "load_bytes: 2, 4, 8 or 16");
    out[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}

// ---------------------------------------------------------------------------
// Registers of a tile.  Both products of a tile are 16x16x32 matrix
// operations whose operands need no move between lanes:
//   S^T = K Q^T: rows are 16 tokens, columns the query heads, K = 32 of the
//     head's values.  Lane (r = lane % 16, g = lane / 16) gives K row r,
//     values 32 step + 8 g .. + 7 (one 16-byte load; 8-bit caches: one
//     16-byte load at 64 u + 16 g covers the steps 2 u and 2 u + 1), and Q
//     the same values of head r.  It gets the scores of head r (= column)
//     and tokens 4 g .. 4 g + 3 of the 16.
//   O^T = V^T P^T: rows are head values, columns the query heads, K = the
//     tile's 32 tokens.  The order of K is free, so the lane's eight are the
//     tokens whose scores it has: 4 g + i and 16 + 4 g + i.  It loads those
//     eight rows of V, values r * PL .. of each (16 lanes read a whole row),
//     and pairs the halves of two tokens' words by byte permutes: operation
//     c has the row values c of every lane's PL = D / 16.
// So the softmax needs lane moves only to join maxima, and the accumulator
// of head r sits with its maximum and sum in the same lanes.
// ---------------------------------------------------------------------------
template <class T, class C, int D>
struct Tile {
  using V = typename ValueType<T, C>::type;
  static constexpr int ES = sizeof(typename C::bits_t);  // bytes of a cached value
  static constexpr int Steps = D / 32;
  static constexpr int PL = D / 16;  // row values of V per lane
  // V's two loads per row: E0 values (the largest power of two that one
  // load holds), then E1
  static constexpr int E0 = ES == 1 ? (PL >= 16 ? 16 : PL >= 8 ? 8 : 4) : (PL >= 8 ? 8 : 4);
  static constexpr int E1 = PL - E0;
  static constexpr int W0 = E0 * ES / 4, W1 = (E1 * ES + 3) / 4;
  static constexpr int KW = D * ES / 4 / 4;  // words of a K row per lane
  static constexpr int Row = D * ES;         // bytes of a cached row

  uint32_t k[2][KW];
  uint32_t v[8][W0 + W1];

  __device__ __forceinline__ void load_k(const uint8_t* const (&base)[2], int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint8_t* row = base[j];
      const uint32_t at = r * Row + (ES == 2 ? 16 * g : 0);
      if constexpr (ES == 2) {
#pragma unroll
        for (int s = 0; s < Steps; ++s) load_bytes<16>(row + at + 64 * s, &k[j][4 * s]);
      } else {
#pragma unroll
        for (int u = 0; u < D / 64; ++u) load_bytes<16>(row + (at + 16 * g) + 64 * u, &k[j][4 * u]);
        if constexpr (D % 64) load_bytes<8>(row + (at + 8 * g) + (D / 64) * 64, &k[j][4 * (D / 64)]);
      }
    }
  }
  __device__ __forceinline__ void load_v(const uint8_t* const (&base)[2], int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint8_t* row = base[e >> 2];
      const uint32_t at = 4 * g * Row;
      load_bytes<E0 * ES>(row + (at + r * (E0 * ES)) + (e & 3) * Row, &v[e][0]);
      if constexpr (E1 > 0)
        load_bytes<E1 * ES>(row + (at + r * (E1 * ES)) + ((e & 3) * Row + 16 * E0 * ES), &v[e][W0]);
    }
  }
  // the head value of operation c in lane row r
  static __device__ __forceinline__ int dim(int r, int c) {
    return c < E0 ? r * E0 + c : 16 * E0 + r * E1 + (c - E0);
  }

  // operand of q.k step s: the values d(s, g, e) of Q or K (see load_k)
  static __device__ __forceinline__ int q_dim(int s, int g) {
    if (ES == 2 || 64 * (s / 2) + 64 > D) return 32 * s + 8 * g;
    return 64 * (s / 2) + 16 * g + 8 * (s % 2);
  }
  __device__ __forceinline__ typename Mma<T>::op k_op(int j, int s) const {
    uint32_t w[4];
    if constexpr (ES == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = k[j][4 * s + i];
    } else {
      Mma<T>::widen(k[j][2 * s], w);
      Mma<T>::widen(k[j][2 * s + 1], w + 2);
    }
    typename Mma<T>::op r;
    __builtin_memcpy(&r, w, 16);
    return r;
  }
  // operand of operations c and c + 1 (c even): tokens e of their row values
  __device__ __forceinline__ void v_ops(int c, typename Mma<V>::op& a, typename Mma<V>::op& b) const {
    uint32_t lo[4], hi[4];
    const int in = c < E0 ? c : c - E0, base = c < E0 ? 0 : W0;
    if constexpr (ES == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = v[2 * i][base + in / 2], y = v[2 * i + 1][base + in / 2];
        lo[i] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(y, x, 0x07060302u);
      }
    } else {
      // bytes (x.c, y.c, x.c+1, y.c+1), then each pair to fp16
      const uint32_t sel = in % 4 == 0 ? 0x05010400u : 0x07030602u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = v[2 * i][base + in / 4], y = v[2 * i + 1][base + in / 4];
        uint32_t w[2];
        Mma<V>::widen(__builtin_amdgcn_perm(y, x, sel), w);
        lo[i] = w[0], hi[i] = w[1];
      }
    }
    __builtin_memcpy(&a, lo, 16);
    __builtin_memcpy(&b, hi, 16);
  }
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A maximum is raised only where a score passes it by more than kSlack (in
// powers of two), so most tiles need no lane moves and no rescaling.
// Probabilities are kept 2^lift times their value, at most 2^(lift + kSlack)
// (Mma::lift).
constexpr float kSlack = 8.0f;

// The parts pass from one workgroup to another, maybe on another die with
// its own L2, by stores and loads that go through to the memory all dies
// share (relaxed atomics of device scope).  Plain stores with a fence would
// write back and drop a die's whole L2 for every workgroup: 2 us each, one
// after the other (1 x 262144 tokens in 512 workgroups: 283 us).
__device__ __forceinline__ void put2(float* p, float a, float b) {
  const uint64_t v = (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get2(const float* p) {
  return __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Infinite values.  A visible one makes its element infinite (NaN where both
// signs or a NaN meet), but times a 16-bit term that is zero or negative, or
// a weight that has become zero, it is NaN.  So an element that came out NaN
// from scores that are numbers is decided again, from the infinite and NaN
// values alone: their sum is what the element is.  (1 x 500 tokens: 9.10 us
// without, 9.28 with the pass over the values inlined among the code that
// every launch fetches, 9.13 with it called; 1 x 262144 tokens of infinite
// values 1.4 ms instead of 0.19.)
__device__ __forceinline__ bool any_nan(const f32x4& o) {
  return __builtin_isunordered(o[0], o[1]) | __builtin_isunordered(o[2], o[3]);
}
__device__ __forceinline__ float not_finite(float v) { return fabsf(v) < INFINITY ? 0.0f : v; }
__device__ __forceinline__ void take_infinite(f32x4& o, const f32x4& s) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (o[i] != o[i] && fabsf(s[i]) == INFINITY) o[i] = s[i];
}
// Values d .. d + 3 of the visible tokens first .. end - 1 (at least one;
// 16-bit caches: E4M3 has no infinity), by one thread, eight tokens in flight
// (past the end the last one again, which changes no such sum).
template <class C, int D>
__device__ __attribute__((noinline)) f32x4 infinite_values(const int32_t* table, const typename C::bits_t* v_cache, int pages,
                                                           int kv_heads, int kh, int page_shift, int first, int end,
                                                           int d) {
  constexpr int kFlight = 8;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int t0 = first; t0 < end; t0 += kFlight) {
    constexpr int kWords = sizeof(typename C::bits_t);  // of four values
    uint32_t v[kFlight][kWords];
    bool in[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int t = min(t0 + j, end - 1);
      const int page = table[t >> page_shift];
      in[j] = page >= 0 && page < pages;
      const int64_t cell = (((int64_t)(in[j] ? page : 0) * kv_heads + kh) << page_shift) + (t & ((1 << page_shift) - 1));
      load_bytes<4 * kWords>(reinterpret_cast<const uint8_t*>(v_cache + cell * D + d), v[j]);
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      if (!in[j]) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = kWords == 2 ? v[j][i / 2] >> (16 * (i % 2)) : v[j][0] >> (8 * i);
        s[i] += not_finite(C::value((typename C::bits_t)w));
      }
    }
  }
  return s;
}
}  // namespace bgg
