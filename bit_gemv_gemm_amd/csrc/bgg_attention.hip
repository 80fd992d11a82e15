// Attention of one new token per sequence over a paged cache:
// s_t = scale q.k_t, out = sum_t e^(s_t) v_t / sum_t e^(s_t).
//
// Every key and value is read once per 16 query heads of its key head, and
// each read value does at most 2 * 16 multiply-adds on the matrix cores, so
// long sequences are bound by the cache's bytes and short ones by the chain
// of dependent loads (length, page numbers, keys; then, where a sequence is
// cut, the parts).  One launch; the tokens are read with running maximum and
// sum, straight from the cache into the operands of the matrix operations.
//
// Measured (one MI355X, which reads 6.14 TB/s; 48 query heads on 8 key heads
// of 128 unless stated): 1 x 262144 tokens f16 186 us (5.76 TB/s), 16 x
// 32768 e4m3 183 us (5.87), 1 x 32768 f16 28.6 us (4.7), 1 x 1024 8.9 us, 1 x
// 64 4.6 us (a kernel that does nothing: 1.7); 16 ragged sequences up to 8000
// tokens, 24 heads on 4 of 256, bf16: 28 us (4.0 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>

#include "bgg_cache.h"
#include "bgg_lowp.h"

using namespace bgg;

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kTokens = 32;  // tokens of a tile: one wave's step
constexpr int kHeads = 16;   // query heads of a workgroup (columns of the products)

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
};

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

// ---------------------------------------------------------------------------
// Which sequence, heads and tokens a workgroup takes.  The visible tokens of
// the batch, in tiles of 32, are cut into chunks of about
// (all tiles) * (head blocks) / target_items tiles, so that a ragged batch
// fills the GPU evenly whatever its longest sequence; every sequence has one
// chunk at least, and its chunks are equal but for rounding.  The lengths
// are on the device, so each wave works this out by itself: lane l sums over
// the sequences [l per, (l + 1) per).  Up to 64 sequences that is one read of
// the lengths; beyond, each wave reads them all several times over, one after
// the other in a lane, and there is a workgroup per sequence and head block
// at least: the schedule's time grows with the square of the batch (40 tokens
// each, 48 heads on 8 of 128 f16: 256 sequences 24 us, 1024 182 us, 4096 2.06
// ms, where their bytes take 8, 31 and 126 us; 500 tokens each: 104 us, 447
// us and 3.0 ms against 86, 346 and 1383).
// ---------------------------------------------------------------------------
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
__device__ __forceinline__ int tiles_of(int lo, int n) {
  return n > lo ? (n - 1) / kTokens - lo / kTokens + 1 : 0;
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

__device__ __forceinline__ bool find_item(const AttnParams& p, int index, Item& it) {
  const int lane = threadIdx.x & 63;
  const int H = p.kv_heads * p.head_blocks;
  const int per = (p.batch + 63) / 64;
  const int b0 = lane * per, b1 = min(p.batch, b0 + per);
  // (the first sequence of the lane stays in registers: up to 64 sequences
  // read their lengths once)
  int lo0 = 0, n0 = 0;
  if (b0 < b1) visible(p, b0, lo0, n0);
  const int t0 = tiles_of(lo0, n0);
  float tiles = (float)t0;
#pragma unroll 1
  for (int b = b0 + 1; b < b1; ++b) {
    int lo, n;
    visible(p, b, lo, n);
    tiles += (float)tiles_of(lo, n);
  }
  // (the sum's fp32 rounding is covered by the factor: the chunks never get
  // more than target_items + batch * H workgroups)
  const float all = wave_add(tiles);
  const float even = fminf(ceilf(all * (float)H / (float)p.target_items * 1.0001f), 1e8f);
  // The last chunk of every sequence is a full workgroup too, so the even
  // size gives a few workgroups more than the GPU takes at once, and they
  // would run alone at the end: a larger size that gives target_items at
  // most, if one up to twice the even size does (16 ragged sequences up to
  // 8000 tokens of 4 x 256 bf16: 280 workgroups 39.8 us, 256 29.7 us).
  // Chunks are counted in the low half, those of sequences with several in
  // the high half.
  int size = 0, upto = 0, mine = 0;
#pragma unroll 1
  for (int k = 8; k <= 16; k += 2) {
    size = max(1, (int)(even * (float)k * 0.125f));
    mine = b0 < b1 ? both_counts(chunks_of(t0, size)) : 0;
#pragma unroll 1
    for (int b = b0 + 1; b < b1; ++b) {
      int lo, n;
      visible(p, b, lo, n);
      mine += both_counts(chunks_of(tiles_of(lo, n), size));
    }
    upto = scan_add(mine);
    if (p.batch * H > p.target_items) break;
    if ((__builtin_amdgcn_readlane(upto, 63) & 0xFFFF) * H <= p.target_items) break;
  }
  size = __builtin_amdgcn_readfirstlane(size);
  const int seq_item = index / H;  // chunks before this one, over all sequences
  const uint64_t past = __ballot((upto & 0xFFFF) > seq_item);
  if (past == 0) return false;
  const int owner = __builtin_ctzll(past);
  int before = __builtin_amdgcn_readlane(upto - mine, owner);
  int b = owner * per;
  if (per > 1) {  // (per <= 64: a sequence per lane)
    const int bb = b + lane;
    int c = 0;
    if (lane < per && bb < p.batch) {
      int lo, n;
      visible(p, bb, lo, n);
      c = both_counts(chunks_of(tiles_of(lo, n), size));
    }
    const int u = scan_add(c) + before;
    const int o = __builtin_ctzll(__ballot((u & 0xFFFF) > seq_item));
    before = __builtin_amdgcn_readlane(u - c, o);
    b += o;
    visible(p, b, lo0, n0);
    it.lo = __builtin_amdgcn_readfirstlane(lo0);
    it.n = __builtin_amdgcn_readfirstlane(n0);
  } else {
    it.lo = __builtin_amdgcn_readlane(lo0, owner);
    it.n = __builtin_amdgcn_readlane(n0, owner);
  }
  const int t = tiles_of(it.lo, it.n), first = it.lo / kTokens;
  it.b = b;
  it.head_block = index % H;
  it.chunks = chunks_of(t, size);
  it.chunk = seq_item - (before & 0xFFFF);
  it.part = (before >> 16) + it.chunk;
  const int each = (t + it.chunks - 1) / it.chunks;
  it.tile = first + it.chunk * each;
  it.tile_end = first + min(t, (it.chunk + 1) * each);
  return true;
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

// Floats of a part: rows of D accumulators, then each row's maximum and sum.
__host__ __device__ constexpr int64_t part_floats(int64_t rows, int64_t D) {
  return (rows * (D + 2) + 3) / 4 * 4;
}
// Chunks of a sequence at most (the items of one sequence and head block,
// about target_items of which there are kMaxItems at most).
constexpr int kMaxItems = 256, kMaxChunks = kMaxItems + 1;

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
__device__ __attribute__((noinline)) f32x4 infinite_values(const int32_t* table, const uint16_t* v_cache, int pages,
                                                           int kv_heads, int kh, int page_shift, int first, int end,
                                                           int d) {
  constexpr int kFlight = 8;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int t0 = first; t0 < end; t0 += kFlight) {
    u32x2 v[kFlight];
    bool in[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int t = min(t0 + j, end - 1);
      const int page = table[t >> page_shift];
      in[j] = page >= 0 && page < pages;
      const int64_t cell = (((int64_t)(in[j] ? page : 0) * kv_heads + kh) << page_shift) + (t & ((1 << page_shift) - 1));
      v[j] = *reinterpret_cast<const u32x2*>(v_cache + cell * D + d);
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      if (!in[j]) continue;
      s[0] += not_finite(C::value((uint16_t)v[j].x));
      s[1] += not_finite(C::value((uint16_t)(v[j].x >> 16)));
      s[2] += not_finite(C::value((uint16_t)v[j].y));
      s[3] += not_finite(C::value((uint16_t)(v[j].y >> 16)));
    }
  }
  return s;
}
// Four accumulators of every part of a sequence.
__device__ __forceinline__ f32x4 infinite_parts(const float* at, int64_t step, int chunks) {
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    const uint64_t a = get2(at + c * step), b = get2(at + c * step + 2);
    s[0] += not_finite(__uint_as_float((uint32_t)a));
    s[1] += not_finite(__uint_as_float((uint32_t)(a >> 32)));
    s[2] += not_finite(__uint_as_float((uint32_t)b));
    s[3] += not_finite(__uint_as_float((uint32_t)(b >> 32)));
  }
  return s;
}

// Values d .. d + 3 of query head h: the accumulator over the sum, rounded
// (0 where no score was above -inf, also if the values there were NaN or inf
// and the accumulator is NaN).
template <class T, class V>
__device__ __forceinline__ void store_out(const AttnParams& p, int b, int h, int D, int d, f32x4 o, float m,
                                          float l, float vs) {
  const bool none = l == 0.0f;
  const float f = vs / l;
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = none ? 0u : (uint32_t)T::bits(o[2 * i] * f) | ((uint32_t)T::bits(o[2 * i + 1] * f) << 16);
  *reinterpret_cast<u32x2*>(p.out + b * p.out_stride + (int64_t)h * D + d) = u32x2{w[0], w[1]};
  if (d == 0 && p.lse)
    p.lse[(int64_t)b * p.q_heads + h] = none ? -INFINITY : (m + (__builtin_amdgcn_logf(l) - Mma<V>::lift)) * kLn2;
}

// The parts of a sequence's chunks (at parts, parts + step, ...) into its
// output: each chunk's weight 2^(m_c - m), then the weighted rows, four
// values (a column) per thread and step; with fewer columns than threads the
// threads also share the chunks out among them.  The maxima and sums and the
// first columns are loaded together, so that up to eight chunks cost one trip
// to memory.  This code runs once, by one workgroup per sequence and head
// block, so its instructions come from memory too: it is kept short by loops
// (unrolled to 16 parts in flight and three columns per thread it took 9 us
// for 32 chunks of 6 x 128).  `lds` holds 32 kMaxChunks floats.
template <class T, class V, int D>
__device__ __forceinline__ void join_parts(const AttnParams& p, const Item& it, const float* parts,
                                           int64_t step, int rows, int heads, int h0, float vs,
                                           float* lds, float* lds16) {
  constexpr int kThreads = 64 * kWaves, kRows = kThreads / 16;  // threads of a head
  constexpr int kFlight = 8;                                    // a thread's parts in flight
  const int tid = threadIdx.x, hr = tid & 15, cr = tid >> 4;
  const int columns = heads * (D / 4);
  const int share = columns >= kThreads ? 1 : kThreads / columns;  // threads per column
  const int part_of = share > 1 ? tid / columns : 0;
  int col = share > 1 ? tid % columns : tid;
  float* weight = lds;                     // [chunks][16]
  float* sum = lds + 16 * kMaxChunks;      // [chunks][16]

  uint64_t a[kFlight][2];
  auto load_flight = [&](int c0, int cb) {
    const float* x = parts + 4 * c0;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int64_t c = min(cb + j * share, it.chunks - 1);
      a[j][0] = get2(x + c * step);
      a[j][1] = get2(x + c * step + 2);
    }
  };
  load_flight(min(col, columns - 1), part_of);

  float mh = -FLT_MAX, lh = 0.0f;
#pragma unroll 1
  for (int c = cr; c < it.chunks; c += kRows) {
    const uint64_t x = get2(parts + c * step + rows * D + 2 * min(hr, heads - 1));
    weight[c * 16 + hr] = __uint_as_float((uint32_t)x);
    sum[c * 16 + hr] = __uint_as_float((uint32_t)(x >> 32));
    mh = fmaxf(mh, __uint_as_float((uint32_t)x));
  }
  lds16[cr * 16 + hr] = mh;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kRows; ++j) mh = fmaxf(mh, lds16[j * 16 + hr]);
#pragma unroll 1
  for (int c = cr; c < it.chunks; c += kRows) {
    const float w = __builtin_amdgcn_exp2f(weight[c * 16 + hr] - mh);
    lh += sum[c * 16 + hr] * w;
    weight[c * 16 + hr] = w;
  }
  float* heads_m = lds16 + 16 * kRows;
  float* heads_l = heads_m + 16;
  if (cr == 0) heads_m[hr] = mh;
  __syncthreads();  // (every maximum is read)
  lds16[cr * 16 + hr] = lh;
  __syncthreads();
  if (cr == 0) {
    lh = 0.0f;
#pragma unroll
    for (int j = 0; j < kRows; ++j) lh += lds16[j * 16 + hr];
    heads_l[hr] = lh;
  }
  __syncthreads();

  // the column of the output, its shares added
  auto store_column = [&](f32x4 o) {
    const int h = col / (D / 4);
    if (__builtin_expect(__any(any_nan(o)), false) && any_nan(o) && heads_l[h] == heads_l[h])
      take_infinite(o, infinite_parts(parts + 4 * col, step, it.chunks));
    store_out<T, V>(p, it.b, h0 + h, D, 4 * (col % (D / 4)), o, heads_m[h], heads_l[h], vs);
  };

  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  int cb = part_of;
  const bool works = part_of < share;
#pragma unroll 1
  while (works && col < columns) {
    const float* w = weight + col / (D / 4);
    // (a part past the last repeats it with weight 0; the select keeps an
    // infinite value there from making a NaN)
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int c = cb + j * share;
      const bool in = c < it.chunks;
      const float wc = w[(in ? c : 0) * 16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = __uint_as_float((uint32_t)(a[j][i / 2] >> (32 * (i % 2))));
        o[i] = in ? fmaf(v, wc, o[i]) : o[i];
      }
    }
    cb += kFlight * share;
    if (cb >= it.chunks) {
      if (share > 1) break;
      store_column(o);
      o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      cb = 0;
      col += kThreads;
      if (col >= columns) break;
    }
    load_flight(col, cb);
  }
  if (share == 1) return;
  __syncthreads();  // (the sums are done with: their place takes the shares)
  if (part_of > 0 && works) *reinterpret_cast<f32x4*>(sum + 4 * (part_of * columns + col)) = o;
  __syncthreads();
  if (part_of > 0) return;
#pragma unroll 1
  for (int j = 1; j < share; ++j) o += *reinterpret_cast<const f32x4*>(sum + 4 * (j * columns + col));
  store_column(o);
}

// One workgroup per item: its waves take the chunk's tiles in turn, each
// with its own maximum, sum and accumulator; joined through LDS, then, where
// a sequence has several chunks, through the workspace: the workgroup that
// arrives last adds the parts in chunk order.
template <class T, class C, int D>
__global__ void __launch_bounds__(64 * kWaves, sizeof(typename C::bits_t) * D > 384 ? 1 : 2) k_paged_attention(AttnParams p) {
  using TL = Tile<T, C, D>;
  using V = typename TL::V;
  constexpr int PL = TL::PL;
  constexpr int RowF = D + 4;  // floats between heads in LDS
  // the waves' accumulators, then join_parts' weights and sums
  constexpr int kRed = kWaves * kHeads * RowF, kJoin = 32 * kMaxChunks;
  __shared__ __attribute__((aligned(16))) float lds[kRed > kJoin ? kRed : kJoin];
  __shared__ float red_m[kWaves][kHeads], red_l[kWaves][kHeads], red_j[64 * kWaves + 32];
  static_assert(4 * 64 * kWaves <= 16 * kMaxChunks, "the shares of the columns fit");
  float(*red)[kHeads][RowF] = reinterpret_cast<float(*)[kHeads][RowF]>(lds);
  __shared__ uint32_t arrived;

  Item it;
  if (!find_item(p, blockIdx.x, it)) return;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kh = it.head_block / p.head_blocks, hb = it.head_block % p.head_blocks;
  const int heads = min(kHeads, p.group - hb * kHeads);
  const int h0 = kh * p.group + hb * kHeads;

  typename Mma<T>::op q[TL::Steps];
#pragma unroll
  for (int s = 0; s < TL::Steps; ++s) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (r < heads)
      load_bytes<16>(reinterpret_cast<const uint8_t*>(p.q + it.b * p.q_stride + (int64_t)(h0 + r) * D + TL::q_dim(s, g)), w);
    __builtin_memcpy(&q[s], w, 16);
  }
  const float factor = p.scale * (p.k_scale ? p.k_scale[kh] : 1.0f) * kLog2e;

  f32x4 acc[PL];
#pragma unroll
  for (int c = 0; c < PL; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -FLT_MAX, l = 0.0f;

  // the page numbers of this wave's tiles, a tile per lane (64 at a time)
  const int32_t* table = p.table + it.b * p.table_stride;
  int page_of[2] = {-1, -1};
  auto load_pages = [&](int tile) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = (tile + kWaves * lane) * kTokens + 16 * j;
      page_of[j] = tile + kWaves * lane < it.tile_end && t < it.n ? table[t >> p.page_shift] : -1;
      if (page_of[j] >= p.pages) page_of[j] = -1;
    }
  };
  struct Place {
    const uint8_t *k[2], *v[2];
    bool ok[2];
  };
  auto place = [&](int step, int tile) {
    Place a;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int page = __builtin_amdgcn_readlane(page_of[j], step & 63);
      a.ok[j] = page >= 0;
      const int t = (tile * kTokens + 16 * j) & ((1 << p.page_shift) - 1);
      const int64_t at = ((((int64_t)(page < 0 ? 0 : page) * p.kv_heads + kh) << p.page_shift) + t) * TL::Row;
      a.k[j] = p.k_cache + at;
      a.v[j] = p.v_cache + at;
    }
    return a;
  };

  TL tl;
  const int first = it.tile + wave;
  Place now;
  if (first < it.tile_end) {
    load_pages(first);
    now = place(0, first);
    tl.load_k(now.k, lane);
    __builtin_amdgcn_sched_barrier(0);  // (keys first: the loop waits for them alone)
    tl.load_v(now.v, lane);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int tile = first, step = 0; tile < it.tile_end; tile += kWaves, ++step) {
    // the tile after this one, or this one again (loads without a branch
    // keep the waits for the loads before them exact)
    const bool more = tile + kWaves < it.tile_end;
    // scores of head r: tokens 16 j + 4 g + i
    f32x4 s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < TL::Steps; ++st) s[j] = Mma<T>::mul(tl.k_op(j, st), q[st], s[j]);
    }
    if (more && ((step + 1) & 63) == 0) load_pages(tile + kWaves);
    const Place next = place(step + more, tile + (more ? kWaves : 0));
    __builtin_amdgcn_sched_barrier(0);
    tl.load_k(next.k, lane);
    __builtin_amdgcn_sched_barrier(0);
    const int t0 = tile * kTokens;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3] * factor;
    if (!(t0 >= it.lo && t0 + kTokens <= it.n && now.ok[0] && now.ok[1])) {
      // hidden tokens: no score, and no value that could be NaN
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = t0 + 16 * (e >> 2) + 4 * g + (e & 3);
        const bool seen = now.ok[e >> 2] && t >= it.lo && t < it.n;
        x[e] = seen ? x[e] : -INFINITY;
#pragma unroll
        for (int w = 0; w < TL::W0 + TL::W1; ++w) tl.v[e][w] = seen ? tl.v[e][w] : 0u;
      }
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
    if (__any(top > m + kSlack)) {
      const float mn = fmaxf(m, column_max(top));
      const float f = __builtin_amdgcn_exp2f(m - mn);
      l *= f;
#pragma unroll
      for (int c = 0; c < PL; ++c) acc[c] *= f;
      m = mn;
    }
    float pr[8], rest[8], none[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pr[e] = __builtin_amdgcn_exp2f(x[e] - m + Mma<V>::lift);
      l += pr[e];
    }
    const typename Mma<V>::op hi = Mma<V>::split(pr, rest), lo = Mma<V>::split(rest, none);
#pragma unroll
    for (int c = 0; c < PL; c += 2) {
      typename Mma<V>::op a, b;
      tl.v_ops(c, a, b);
      acc[c] = Mma<V>::mul(a, hi, acc[c]);
      acc[c] = Mma<V>::mul(a, lo, acc[c]);
      acc[c + 1] = Mma<V>::mul(b, hi, acc[c + 1]);
      acc[c + 1] = Mma<V>::mul(b, lo, acc[c + 1]);
    }
    __builtin_amdgcn_sched_barrier(0);
    tl.load_v(next.v, lane);
    __builtin_amdgcn_sched_barrier(0);
    now = next;
  }

  // the waves' parts
  l = column_sum(l);
  if (g == 0) red_m[wave][r] = m, red_l[wave][r] = l;
  __syncthreads();
  float mw = red_m[0][r];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) mw = fmaxf(mw, red_m[w][r]);
  if (r < heads) {
    const float f = __builtin_amdgcn_exp2f(m - mw);
#pragma unroll
    for (int c = 0; c < PL; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][r][TL::dim(4 * g + i, c)] = acc[c][i] * f;
  }
  __syncthreads();
  // thread i takes four values of a head
  const float vs = p.v_scale ? p.v_scale[kh] : 1.0f;
  const int H = p.kv_heads * p.head_blocks, rows = min(kHeads, p.group);
  const int64_t slot = part_floats(rows, D);
  float* part = p.parts + ((int64_t)it.part * H + it.head_block) * slot;
  const int columns = heads * (D / 4);
  for (int i = threadIdx.x; i < columns; i += 64 * kWaves) {
    const int h = i / (D / 4), d = 4 * (i % (D / 4));
    float mh = red_m[0][h], lh = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mh = fmaxf(mh, red_m[w][h]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      lh += red_l[w][h] * __builtin_amdgcn_exp2f(red_m[w][h] - mh);
      o += *reinterpret_cast<const f32x4*>(&red[w][h][d]);
    }
    if constexpr (sizeof(typename C::bits_t) == 2)
      if (__builtin_expect(__any(any_nan(o)), false) && any_nan(o) && lh == lh) {
        const int end = (int)min((int64_t)it.n, (int64_t)it.tile_end * kTokens);
        take_infinite(o, infinite_values<C, D>(table, reinterpret_cast<const uint16_t*>(p.v_cache), p.pages, p.kv_heads, kh,
                                               p.page_shift, max(it.lo, it.tile * kTokens), end, d));
      }
    if (it.chunks == 1) {
      store_out<T, V>(p, it.b, h0 + h, D, d, o, mh, lh, vs);
    } else {
      put2(part + h * D + d, o[0], o[1]);
      put2(part + h * D + d + 2, o[2], o[3]);
      if (d == 0) put2(part + rows * D + 2 * h, mh, lh);
    }
  }
  if (it.chunks == 1) return;

  // every thread's stores of this part have reached the shared memory (their
  // count is back to zero) before its arrival shows; the last arrival reads
  // the others' after it
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  uint32_t* counter = p.counters + (it.part - it.chunk) * H + it.head_block;
  if (threadIdx.x == 0)
    arrived = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (arrived != (uint32_t)it.chunks - 1) return;
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  join_parts<T, V, D>(p, it, part - (int64_t)it.chunk * H * slot, H * slot, rows, heads, h0, vs,
                   lds, red_j);
}

// ---------------------------------------------------------------------------
// plan and launch
// ---------------------------------------------------------------------------

struct AttnPlan {
  int64_t heads;  // head blocks of all key heads
  int64_t target, items, parts;
  uint64_t total_bytes;
};
// The arrival counters sit at the start of every workspace, whatever the
// call's shape, so that one workspace serves any sequence of calls: a
// sequence of several chunks counts in the word of its first part.
constexpr uint64_t kCounterBytes = BGG_ATTENTION_COUNTER_BYTES;
static_assert(2 * kMaxItems * 4 <= kCounterBytes, "a counter per part");

AttnPlan plan_attention(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  AttnPlan p;
  p.heads = c->kv_heads * ceil_div(q_heads / c->kv_heads, kHeads);
  // one workgroup per CU: each one more per CU costs its own start and part
  // (1 x 262144 tokens f16: 1, 2, 3, 4 per CU 189, 193, 200, 208 us; 16
  // ragged sequences up to 8000 tokens of 4 x 256 bf16: 39, 44, 51, 59 us)
  p.target = std::min<int64_t>(device_cus(), kMaxItems);
  p.items = p.target + batch * p.heads;
  // (a sequence of n > 1 chunks has more than (n - 1) >= n / 2 full ones)
  p.parts = 2 * kMaxItems;  // (whatever the device, so that the size does not depend on it)
  p.total_bytes = kCounterBytes + align256(
      4 * (uint64_t)(p.parts * part_floats(std::min<int64_t>(kHeads, q_heads / c->kv_heads), c->head_dim)));
  return p;
}

template <class T, class C>
void launch_dim(const AttnParams& p, int64_t items, int64_t head_dim, hipStream_t s) {
  const dim3 grid((unsigned)items), block(64 * kWaves);
  switch (head_dim) {
    case 64: hipLaunchKernelGGL((k_paged_attention<T, C, 64>), grid, block, 0, s, p); break;
    case 96: hipLaunchKernelGGL((k_paged_attention<T, C, 96>), grid, block, 0, s, p); break;
    case 128: hipLaunchKernelGGL((k_paged_attention<T, C, 128>), grid, block, 0, s, p); break;
    case 192: hipLaunchKernelGGL((k_paged_attention<T, C, 192>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((k_paged_attention<T, C, 256>), grid, block, 0, s, p); break;
  }
}

}  // namespace

extern "C" {

size_t bgg_attention_workspace_size(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  if (check_cache(c) != BGG_OK || q_heads < 1 || q_heads > kMaxQHeads || q_heads % c->kv_heads ||
      batch < 1 || batch > kMaxBatch)
    return 0;
  return (size_t)plan_attention(c, q_heads, batch).total_bytes;
}

bgg_status bgg_paged_attention(const bgg_cache_desc* c, const bgg_attention_args* a, void* stream) {
  bgg_status st = check_attention(c, a);
  if (st) return st;
  if (a->batch == 0) return BGG_OK;
  const AttnPlan plan = plan_attention(c, a->q_heads, a->batch);
  if (a->workspace_bytes < plan.total_bytes)
    return fail(BGG_ERR_BUFFER, "bgg_paged_attention: workspace has %zu bytes, needs %llu",
                a->workspace_bytes, (unsigned long long)plan.total_bytes);
  AttnParams p{};
  p.q = (const uint16_t*)a->q_dev;
  p.out = (uint16_t*)a->out_dev;
  p.q_stride = a->q_stride;
  p.out_stride = a->out_stride;
  p.lse = a->lse_dev;
  p.k_cache = (const uint8_t*)a->k_cache_dev;
  p.v_cache = (const uint8_t*)a->v_cache_dev;
  p.k_scale = a->k_scale_dev;
  p.v_scale = a->v_scale_dev;
  p.table = a->page_table_dev;
  p.table_stride = a->table_stride;
  p.lengths = a->lengths_dev;
  p.window = a->window;
  p.counters = (uint32_t*)a->workspace;
  p.parts = (float*)((uint8_t*)a->workspace + kCounterBytes);
  p.max_tokens = (int)(a->table_width * c->page_size);
  p.scale = a->scale;
  p.pages = (int)c->pages;
  p.batch = (int)a->batch;
  p.q_heads = (int)a->q_heads;
  p.kv_heads = (int)c->kv_heads;
  p.group = (int)(a->q_heads / c->kv_heads);
  p.head_blocks = (int)ceil_div(p.group, kHeads);
  p.page_shift = __builtin_ctzll((unsigned long long)c->page_size);
  p.target_items = (int)plan.target;
  hipStream_t s = (hipStream_t)stream;
  const bool e4m3 = c->type == BGG_TYPE_E4M3;
  if (a->type == BGG_TYPE_F16) {
    if (e4m3)
      launch_dim<F16, E4M3>(p, plan.items, c->head_dim, s);
    else
      launch_dim<F16, F16>(p, plan.items, c->head_dim, s);
  } else {
    if (e4m3)
      launch_dim<BF16, E4M3>(p, plan.items, c->head_dim, s);
    else
      launch_dim<BF16, BF16>(p, plan.items, c->head_dim, s);
  }
  return hip_check("bgg_paged_attention");
}

}  // extern "C"
