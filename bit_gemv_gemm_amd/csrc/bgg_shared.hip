// The shared part of bgg_shared_attention: groups of sequences whose first
// pages are the same read those pages once.  With the members' query heads of
// a key head as rows, it is a product of many rows with the prefix: for a
// chunk of tokens t and row r, m_r = max s_rt, l_r = sum 2^(s_rt - m_r),
// o_r = sum 2^(s_rt - m_r) v_t with s = log2(e) scale q_r k_t, in fp32, which
// k_paged_attention joins with the sequence's own tokens.  Bound by the matrix
// and vector units instead of the cache's bytes as soon as a group has more
// than a few members.
//
// A workgroup takes up to 256 rows of a key head (128 of wide heads) and a
// chunk of the prefix; keys and values go from the cache to LDS once for all
// its waves.  64 sequences of 48/8 heads of 128 behind 32768 tokens of f16: 93
// us, of which 7.5 pass until the first tiles are there and 4 with the parts at
// the end; 256 sequences in two groups behind 5328 and 4112 tokens of bf16
// (32/8): 51 us.  The matrix units are busy 48 and 34 % of the time and the
// vector units 54 and 46 %, and the clock falls to about 1.8 GHz under them.
// (Where both sides of a choice are given below, they were measured with
// probabilities of one term.)
//
// What grows with the groups is the schedule: every workgroup works it out by
// itself, a part of them only to find nothing left, and one at a time runs on a
// CU.  us, of 32/8 heads of 128 f16 behind 1024 tokens, with bgg_paged_attention
// of the same batch: 32, 64, 128, 512 groups of 8 sequences 53, 115, 230, 1110
// (100, 225, 507, 3420); 64, 512, 2048 groups of 2 77, 690, 6200 (64, 628, 3800);
// 64, 256, 1024, 4096 groups of one 69, 289, 1540, 22700 (45, 198, 785, 4280).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bgg_paged.h"
#include "bgg_shared.h"

using namespace bgg;

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 32x32x16 matrix operations: the same values a cycle as 16x16x32 in half the
// instructions (products and exponentials of a tile alone, two waves on a
// SIMD: 1447 cycles against 1551; the kernel's cases 2 to 5 % faster but for
// one of many partly hidden tiles, 27.0 against 28.1 us).
__device__ __forceinline__ f32x16 mul32(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mul32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zeros() {
  f32x16 v;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  return v;
}
// Over the two lanes of a row.
__device__ __forceinline__ float row_max(float v) {
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_sum(float v) {
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

constexpr int kGroupsMax = (int)kMaxBatch;

// (the last tile of the longest table ends at 2^31, behind every token: cut)
__device__ __forceinline__ int first_token(int tile) { return (int)min((uint32_t)tile * kTokens, 0x7FFFFFFFu); }

// The shape of the kernel's work.
template <class T, class C, int D>
struct PrefixShape {
  using TL = Tile<T, C, D>;
  static constexpr int Row = TL::Row;
  // Eight waves, two on a SIMD, so that one's matrix operations run beside
  // the other's exponentials; wide heads do not fit their registers.
  static constexpr int Waves = D <= 128 ? 8 : 4, WaveBits = D <= 128 ? 3 : 2;
  static constexpr int Rows = 32;  // of a wave (queries, accumulators)
  static constexpr int Steps = D / 16, PL = D / 32;  // matrix operations of the scores, of 16 tokens' values
  // The operands of a tile (in lane l: r = l % 32, h = l / 32):
  //   S^T = K Q^T: rows are the tile's 32 tokens, columns 32 query rows, and
  //     lane (r, h) gives values q_dim .. + 7 of token r and of row r.  It
  //     gets the scores of row r at tokens 8 (i / 4) + 4 h + i % 4, i < 16.
  //   O^T = V^T P^T: rows are 32 of the head's values, columns the rows; the
  //     order of the tokens is free, so operation j of the two takes those of
  //     the scores 8 j .. 8 j + 7, and lane (r, h) gets values 8 (i / 4) +
  //     4 h + i % 4 of row r.
  static __device__ __forceinline__ int q_dim(int s, int h) {
    return TL::ES == 2 ? 16 * s + 8 * h : 32 * (s / 2) + 16 * h + 8 * (s % 2);
  }
  static constexpr int RowF = D + 4;  // floats of a row of the parts: values, maximum, sum
  // tiles of a step; the keys and values of two steps take up to 128 KB of LDS
  static constexpr int Subs = Waves / 2;
  // Four waves fetch them, a tile each (two a step: half a tile).  Of eight
  // they are the ones whose instructions the SIMDs prefer: the others work
  // while these stand in the queue of the loads.
  static constexpr int Halves = Subs / 2;  // half tiles of a fetching wave
  static constexpr int Least = 2;  // row waves at least
  static constexpr int TileBytes = kTokens * Row;
  static constexpr int Pieces = Row / 16;                // 16-byte pieces of a row
  static constexpr int Loads = (16 * Pieces + 63) / 64;  // of the keys (and the values) of half a tile
  // In LDS, piece q of row r lies at piece q ^ mix(r) of the row, so that what
  // is read together lies in different banks (256 bytes hold all banks once):
  // of the keys, piece q of 16 rows; of the values, 64 bytes of rows 4 n .. 4 n
  // + 3, or 32 bytes (8-bit) of those and of the rows 8 behind them.  (With a
  // mix for other reads half of LDS' cycles were conflicts: 79 us, not 76.5.)
  static __device__ __forceinline__ int mix_k(int r) {
    return Pieces % 16 == 0 ? r & 15 : Pieces % 8 == 0 ? (r >> 1) & 7 : Pieces % 4 == 0 ? (r >> 2) & 3 : (r >> 3) & 1;
  }
  static __device__ __forceinline__ int mix_v(int r) {
    if (TL::ES == 2) return Pieces % 16 == 0 ? 4 * (r & 3) : Pieces % 8 == 0 ? 4 * ((r >> 1) & 1) : 0;
    return 2 * (Pieces % 16 == 0 ? (r & 3) | ((r >> 1) & 4) : Pieces % 8 == 0 ? ((r >> 1) & 1) | ((r >> 2) & 2) : Pieces % 4 == 0 ? (r >> 3) & 1 : 0);
  }
};

template <int MOVE, int ROWS>
__device__ __forceinline__ int max_from(int v) {
  return max(v, __builtin_amdgcn_update_dpp(0, v, MOVE, ROWS, 0xF, false));
}

// The batch, in LDS: sequence b has n[b] tokens and shares pages[b] pages
// (of which a group's first counts); group g has the sequences start[g] ..
// start[g + 1] - 1, which see tokens lo .. hi - 1 of its prefix.
struct Batch {
  int *n, *pages;  // [kGroupsMax]
  int *lo, *hi;    // [kGroupsMax]
  uint16_t* start;  // [kGroupsMax + 1]

  __device__ __forceinline__ int prefix(const AttnParams& p, int g) const { return pages[start[g]] << p.page_shift; }
  __device__ __forceinline__ int first_seen(const AttnParams& p, int b) const {
    return p.window > 0 && n[b] > p.window ? n[b] - (int)p.window : 0;
  }
  // Largest g <= G - 1 with start[g] <= b (or 0).
  __device__ __forceinline__ int group_of(int G, int b) const {
    int g = 0, m = G;
#pragma unroll 1
    while (m > 1) {
      const int half = m >> 1;
      const bool right = start[g + half] <= b;
      g = right ? g + half : g;
      m = right ? m - half : half;
    }
    return g;
  }
};

template <int WAVES>
__device__ __forceinline__ void read_batch(const AttnParams& p, const Batch& s) {
  constexpr int kThreads = 64 * WAVES;
  const int tid = threadIdx.x, G = p.groups;
  for (int b = tid; b < p.batch; b += kThreads) {
    s.n[b] = min(max(p.lengths[b], 0), p.max_tokens);
    s.pages[b] = min(max(p.shared_pages[b], 0), p.max_tokens >> p.page_shift);
  }
  for (int g = tid; g < G; g += kThreads) s.lo[g] = 0x7FFFFFFF, s.hi[g] = 0;
  // starts below an earlier one count as that one, so that no sequence is in
  // two groups whatever the caller's array holds
  if (tid < 64) {
    int before = 0;
    for (int g0 = 0; g0 <= G; g0 += 64) {
      const int g = g0 + tid;
      int v = g <= G ? min(max(p.group_starts[g], 0), p.batch) : 0;
      v = max_from<0x111, 0xF>(v);
      v = max_from<0x112, 0xF>(v);
      v = max_from<0x114, 0xF>(v);
      v = max_from<0x118, 0xF>(v);
      v = max_from<0x142, 0xA>(v);
      v = max_from<0x143, 0xC>(v);
      v = max(v, before);
      if (g <= G) s.start[g] = (uint16_t)v;
      before = __builtin_amdgcn_readlane(v, 63);
    }
  }
  __syncthreads();
  for (int b = s.start[0] + tid; b < s.start[G]; b += kThreads) {
    const int g = s.group_of(G, b), lo = s.first_seen(p, b), n = min(s.n[b], s.prefix(p, g));
    if (lo < n) {
      atomicMin(&s.lo[g], lo);
      atomicMax(&s.hi[g], n);
    }
  }
  __syncthreads();
}

// How a group's prefix is cut: into blocks of rows and chunks of tokens.
struct Cut {
  int tiles, rows;
  int wave_bits;  // 2^wave_bits waves of a workgroup on different rows, the others on other tokens
  int blocks, chunks;
};
// Row waves share the tiles that LDS holds, so there are as many as fit the
// rows with at most a fifth of them empty (396 rows, bf16 heads of 128: eight
// waves in two workgroups, 19 % empty, against two in seven: 256 sequences
// 45.9 and 50.8 us; 384 rows: four in three against eight in two, a quarter
// empty: 79.6 and 90 us; both with the 16x16x32 operations of before).
template <class S>
__device__ __forceinline__ Cut cut_of(const AttnParams& p, const Batch& s, int g) {
  Cut c;
  c.tiles = tiles_of(s.lo[g], s.hi[g]);
  c.rows = (s.start[g + 1] - s.start[g]) * p.group;
  const int units = (c.rows + S::Rows - 1) / S::Rows;  // waves that work
  c.wave_bits = S::WaveBits;
#pragma unroll
  for (int i = 0; i < S::WaveBits; ++i) {
    const int w = 1 << c.wave_bits, padded = (units + w - 1) >> c.wave_bits << c.wave_bits;
    if (c.wave_bits > 1 && padded * 4 > units * 5) --c.wave_bits;
  }
  c.blocks = (units + (1 << c.wave_bits) - 1) >> c.wave_bits;
  return c;
}
// Chunks, and the tiles of each, at a size of items in tiles times row waves:
// a tile or more for every stream of tokens.  (Nothing weighs the parts against
// that: 64 sequences of 16 heads on one key head behind 2048 tokens have 32
// chunks of two tiles, 35 MB of parts, and take 35 us, bgg_paged_attention 15;
// 128 of 32/8 heads 46 and 85.)
template <class S>
__device__ __forceinline__ void cut_tiles(Cut& c, int size) {
  const int streams = S::WaveBits - c.wave_bits;
  const int each = (((size - 1) >> S::WaveBits) + 1) << streams;
  c.chunks = (int)((uint32_t)(c.tiles + each - 1) / (uint32_t)each);
}

struct PrefixItem {
  int group, kh, block, chunk, row;  // row: the group's first row of the parts
  int wave_bits;
  int tile, tile_end;
};

// The item of workgroup `index`, and in `base`, if given, the first row of
// every group's parts and the size of an item.  Every wave works it out by
// itself.
template <class S>
__device__ __forceinline__ bool find_prefix(const AttnParams& p, const Batch& s, int index, PrefixItem& it, int* base,
                                            int* size_out) {
  const int lane = threadIdx.x & 63, G = p.groups;
  const int per = (G + 63) / 64, g0 = min(G, lane * per), g1 = min(G, g0 + per);
  float work = 0.0f;
  Cut one{0, 0, 0, 0, 0};  // the lane's only group's, if there are not more
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    const Cut c = one = cut_of<S>(p, s, g);
    work += (float)c.tiles * (float)(c.blocks << c.wave_bits);
  }
  const float even = fminf(ceilf(wave_add(work) * (float)p.kv_heads / (float)p.prefix_target * 1.0001f), 1e8f);
  int size = 0, mine = 0, upto = 0, rows = 0;
#pragma unroll 1
  for (int k = 32; k <= 64; ++k) {
    size = max(1, (int)(even * (float)k * 0.03125f));
    mine = rows = 0;
    int least = 0;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      Cut c = one;
      if (per > 1) c = cut_of<S>(p, s, g);
      cut_tiles<S>(c, size);
      mine += c.chunks * c.blocks;
      least += c.chunks ? c.blocks : 0;
      rows += c.chunks * p.kv_heads * c.rows;
    }
    upto = scan_add(mine);
    if (__builtin_amdgcn_readlane(upto, 63) * p.kv_heads <= p.prefix_target) break;
    if (wave_add((float)least) * (float)p.kv_heads > (float)p.prefix_target) break;  // (no size is large enough)
  }
  size = __builtin_amdgcn_readfirstlane(size);
  int row = scan_add(rows) - rows;  // rows of the parts before this lane's groups
  if (base) {
    *size_out = size;
    if (threadIdx.x < 64) {
      int r = row;
#pragma unroll 1
      for (int g = g0; g < g1; ++g) {
        Cut c = cut_of<S>(p, s, g);
        cut_tiles<S>(c, size);
        base[g] = r;
        r += c.chunks * p.kv_heads * c.rows;
      }
    }
  }
  const int at = index / p.kv_heads;
  const uint64_t past = __ballot(upto > at);
  if (past == 0) return false;
  const int owner = __builtin_ctzll(past);
  // the owner's groups, by every lane alike
  int first = __builtin_amdgcn_readlane(upto - mine, owner);
  row = __builtin_amdgcn_readlane(row, owner);
  int g = owner * per;
  Cut c;
#pragma unroll 1
  for (;; ++g) {
    c = cut_of<S>(p, s, g);
    cut_tiles<S>(c, size);
    if (at < first + c.chunks * c.blocks) break;
    first += c.chunks * c.blocks;
    row += c.chunks * p.kv_heads * c.rows;
  }
  it.group = __builtin_amdgcn_readfirstlane(g);
  it.kh = index % p.kv_heads;
  it.row = __builtin_amdgcn_readfirstlane(row);
  it.wave_bits = __builtin_amdgcn_readfirstlane(c.wave_bits);
  const int local = at - first;
  it.block = __builtin_amdgcn_readfirstlane(local % c.blocks);
  it.chunk = __builtin_amdgcn_readfirstlane(local / c.blocks);
  const int t0 = s.lo[g] / kTokens;
  const int streams = S::WaveBits - c.wave_bits;
  const int each = ((int)((uint32_t)(c.tiles + c.chunks - 1) / (uint32_t)c.chunks) + (1 << streams) - 1) >> streams << streams;
  it.tile = __builtin_amdgcn_readfirstlane(t0 + min(c.tiles, it.chunk * each));
  it.tile_end = __builtin_amdgcn_readfirstlane(t0 + min(c.tiles, (it.chunk + 1) * each));
  return true;
}

// The schedule of the sequences' own tokens (one workgroup): chunks as
// bgg_paged_attention cuts them, an entry each.
template <class S>
__device__ __forceinline__ void plan_own(const AttnParams& p, const Batch& s, const int* base, int size_of_prefix,
                                         int* scratch) {
  constexpr int kThreads = 64 * S::Waves;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int H = p.kv_heads * p.head_blocks, G = p.groups;
  const int per = (p.batch + kThreads - 1) / kThreads, b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  auto own = [&](int b, int& lo, int& n) {
    n = s.n[b];
    lo = s.first_seen(p, b);
    const int g = s.group_of(G, b);
    if (s.start[g] <= b && b < s.start[g + 1]) lo = max(lo, s.prefix(p, g));
  };
  // (by one wave a sequence of up to two shares stays whole: two items side by
  // side gain less than their join costs)
  const int whole = p.own_target > p.target_items ? 2 : 1;
  auto own_chunks = [&](int tiles, int size) {
    return tiles <= whole * size ? 1 : chunks_of(tiles, max(size, (tiles + p.own_chunks - 1) / p.own_chunks));
  };
  float* const sums = reinterpret_cast<float*>(scratch);
  float tiles = 0.0f;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    int lo, n;
    own(b, lo, n);
    tiles += (float)tiles_of(lo, n);
    SharedSeq q{0, 0, 0};
    const int g = s.group_of(G, b);
    if (s.start[g] <= b && b < s.start[g + 1]) {
      Cut c = cut_of<S>(p, s, g);
      cut_tiles<S>(c, size_of_prefix);
      q.chunks = c.chunks;
      q.rows = c.rows;
      q.row = base[g] + (b - s.start[g]) * p.group;
    }
    p.seqs[b] = q;
  }
  tiles = wave_add(tiles);
  if (lane == 0) sums[wave] = tiles;
  __syncthreads();
  float all = 0.0f;
#pragma unroll
  for (int w = 0; w < S::Waves; ++w) all += sums[w];
  __syncthreads();
  const float even = fminf(ceilf(all * (float)H / (float)p.own_target * 1.0001f), 1e8f);
  int size = 0, mine = 0, before = 0;
#pragma unroll 1
  for (int k = 8; k <= 16; k += 2) {
    size = max(1, (int)(even * (float)k * 0.125f));
    mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      int lo, n;
      own(b, lo, n);
      mine += both_counts(own_chunks(tiles_of(lo, n), size));
    }
    const int upto = scan_add(mine);
    if (lane == 63) scratch[wave] = upto;
    __syncthreads();
    before = upto - mine;
    int total = 0;
#pragma unroll
    for (int w = 0; w < S::Waves; ++w) {
      if (w < wave) before += scratch[w];
      total += scratch[w];
    }
    __syncthreads();
    if (tid == 0) *p.own_count = total & 0xFFFF;
    if (p.batch * H > p.own_target || (total & 0xFFFF) * H <= p.own_target) break;
  }
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    OwnItem it;
    own(b, it.lo, it.n);
    const int t = tiles_of(it.lo, it.n), first = it.lo / kTokens, chunks = own_chunks(t, size);
    const int each = (t + chunks - 1) / chunks;
    it.b = b;
    it.chunks = chunks;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      it.chunk = c;
      it.part = (before >> 16) + c;
      it.tile = first + c * each;
      it.tile_end = first + min(t, (c + 1) * each);
      p.own_items[(before & 0xFFFF) + c] = it;
    }
    before += both_counts(chunks);
  }
}

// Halves of a word whose exponent is all ones to 0; `found` if there is one.
template <class V>
__device__ __forceinline__ uint32_t finite_halves(uint32_t w, bool& found) {
  constexpr uint32_t e = (uint32_t)V::exponent;
  const bool lo = (w & e) == e, hi = (w & (e << 16)) == (e << 16);
  found |= lo | hi;
  return (lo ? 0u : w & 0xFFFFu) | (hi ? 0u : w & 0xFFFF0000u);
}

// Halves of a word times 0: NaN where they are infinite or NaN.
template <class T>
__device__ __forceinline__ uint32_t not_finite_halves(uint32_t w) {
  constexpr uint32_t e = (uint32_t)T::exponent;
  return ((w & e) == e ? 0x7FFFu : 0u) | ((w & (e << 16)) == (e << 16) ? 0x7FFF0000u : 0u);
}

constexpr int at_least(int a, int b) { return a > b ? a : b; }

// 16 bytes per lane from base + from to LDS, lane l's at `to` + 16 l, without
// registers.  In assembly, so that the compiler, which does not see what is
// read while they are in flight, does not wait for every load before it reads
// LDS; landed_barrier is what waits.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // (that m0 is reserved: the compiler writes it where it needs it)
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(from), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop
// All but the youngest N of this wave's loads have landed (those to LDS
// included) and its LDS reads are done, and so for the other waves.
template <int N>
__device__ __forceinline__ void landed_barrier() {
  static_assert(N < 64, "the counter has six bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The keys and values of a step's tiles go from the cache to LDS without
// registers, a step or two ahead, four waves a quarter each; all the waves
// that work on the same tokens read them from there.  Probabilities are a sum
// of two 16-bit terms in the products with the values, as in
// bgg_paged_attention (Mma::split).  The second term doubles these products:
// one alone takes 78.8 us in the place of 93 for 64 sequences behind 32768
// tokens and 43.9 in the place of 51.4 for 256 in two groups, but leaves every
// probability half a step of 16 bits off (up to 2^-8 of its value for bf16), by
// which a sequence's result would change with the call that computes it.
template <class T, class C, int D>
__global__ void __launch_bounds__((64 * PrefixShape<T, C, D>::Waves)) k_shared_prefix(AttnParams p) {
  using TL = Tile<T, C, D>;
  using V = typename TL::V;
  using S = PrefixShape<T, C, D>;
  constexpr int PL = S::PL, Steps = S::Steps, RowF = S::RowF, Row = S::Row, Subs = S::Subs, Waves = S::Waves;
  constexpr int kThreads = 64 * Waves;
  constexpr int kKeys = Subs * S::TileBytes, kBuf = 2 * kKeys;  // a step's keys, then its values
  // two buffers; before and after the loop other uses
  constexpr int kPlan = 24 * kGroupsMax + 16, kRed = 4 * Waves * S::Rows * RowF;
  __shared__ __attribute__((aligned(16))) uint8_t lds[at_least(2 * kBuf, at_least(kPlan, kRed))];
  __shared__ float red_m[Waves * S::Rows];
  __shared__ int scratch[Waves];
  __shared__ __attribute__((aligned(16))) float special[D];  // sums of infinite and NaN values
  __shared__ __attribute__((aligned(8))) uint8_t has_page[2][2 * S::Subs];  // of a step's buffer: half a tile each

  int* const plan = (int*)lds;
  const Batch batch{plan, plan + kGroupsMax, plan + 2 * kGroupsMax, plan + 3 * kGroupsMax, (uint16_t*)(plan + 4 * kGroupsMax)};
  int* const base = plan + 5 * kGroupsMax;  // (the starts take half of the words before, and one value more)
  read_batch<Waves>(p, batch);
  PrefixItem it;
  if (blockIdx.x == 0) {
    int size;
    find_prefix<S>(p, batch, 0, it, base, &size);
    __syncthreads();
    plan_own<S>(p, batch, base, size, scratch);
    return;
  }
  if (!find_prefix<S>(p, batch, blockIdx.x - 1, it, nullptr, nullptr)) return;
  const int lane = threadIdx.x & 63, r = lane & 31, half_of = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kh = it.kh;
  const int s0 = batch.start[it.group], members = batch.start[it.group + 1] - s0, rows = members * p.group;
  const int prefix = batch.prefix(p, it.group);
  const int lo_all = batch.lo[it.group], hi_all = batch.hi[it.group];
  // rows: those of wave % row_waves; tokens: those of wave / row_waves
  const int row_waves = 1 << it.wave_bits, streams = Waves >> it.wave_bits, stream = wave >> it.wave_bits;
  const int row0 = ((it.block << it.wave_bits) + (wave & (row_waves - 1))) * S::Rows;

  // --- from the cache to LDS: the wave's half tiles of a step; the pages of
  // 64 steps at a time, one per lane
  const int32_t* table = p.table + s0 * p.table_stride;
  const int steps = (it.tile_end - it.tile + Subs - 1) / Subs;
  int page_of[S::Halves];
  const bool fetches = wave < 4;
  auto load_pages = [&](int step) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < S::Halves; ++j) {
      const int half = wave * S::Halves + j, tile = it.tile + (step + lane) * Subs + half / 2;
      const int t = tile * kTokens + 16 * (half & 1);
      page_of[j] = tile < it.tile_end && t < hi_all ? table[t >> p.page_shift] : -1;
      if (page_of[j] >= p.pages) page_of[j] = -1;
    }
  };
  if (fetches) load_pages(0);

  // the lane's row: the tokens it sees (a row past the last reads its queries)
  const int member = min((row0 + r) / p.group, members - 1), head = row0 + r < rows ? row0 + r - member * p.group : 0;
  const int lo = batch.first_seen(p, s0 + member), hi = min(batch.n[s0 + member], prefix);
  // a row that sees nothing of the item's tokens (an unused sequence, a
  // window) does not keep the others from the fast path: it is emptied at the
  // end instead
  const bool none = row0 + r >= rows || max(lo, first_token(it.tile)) >= min(hi, first_token(it.tile_end));
  int lo_max = none ? 0 : lo, hi_min = none ? 0x7FFFFFFF : hi;
  // over the rows (the same in both lanes of a row)
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    lo_max = max(lo_max, __shfl_xor(lo_max, s));
    hi_min = min(hi_min, __shfl_xor(hi_min, s));
  }
  lo_max = __builtin_amdgcn_readfirstlane(lo_max);
  hi_min = __builtin_amdgcn_readfirstlane(hi_min);
  __syncthreads();  // (the batch is read: its place takes the tiles)

  int from_k[S::Loads], from_v[S::Halves][S::Loads];  // where in a half's tokens a lane's piece of each load is
#pragma unroll
  for (int i = 0; i < S::Loads; ++i) {
    const int piece = 64 * i + lane, row = piece / S::Pieces, at = piece % S::Pieces;
    from_k[i] = row * Row + 16 * (at ^ S::mix_k(row));
#pragma unroll
    for (int j = 0; j < S::Halves; ++j)
      from_v[j][i] = row * Row + 16 * (at ^ S::mix_v(16 * ((wave * S::Halves + j) & 1) + row));
  }
  const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds + wave * (S::Halves * 16 * Row);
  // keys and values of a step into buffer step % 2
  auto fetch = [&](int step) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < S::Halves; ++j) {
      const int half = wave * S::Halves + j, page = __builtin_amdgcn_readlane(page_of[j], step & 63);
      const int t = ((it.tile + step * Subs + half / 2) * kTokens + 16 * (half & 1)) & ((1 << p.page_shift) - 1);
      const int64_t at = ((((int64_t)(page < 0 ? 0 : page) * p.kv_heads + kh) << p.page_shift) + t) * Row;
      const uint32_t to = lds_at + (step & 1) * kBuf + j * (16 * Row);
#pragma unroll
      for (int i = 0; i < S::Loads; ++i)
        if (16 * S::Pieces % 64 == 0 || 64 * i + lane < 16 * S::Pieces) load_to_lds(p.k_cache + at, from_k[i], to + 1024 * i);
#pragma unroll
      for (int i = 0; i < S::Loads; ++i)
        if (16 * S::Pieces % 64 == 0 || 64 * i + lane < 16 * S::Pieces)
          load_to_lds(p.v_cache + at, from_v[j][i], to + kKeys + 1024 * i);
      if (lane == 0) has_page[step & 1][half] = page >= 0;
    }
  };
  if (fetches && steps > 0) fetch(0);

  // the queries, while those are on their way
  // (the factor is kept positive, for the maxima: a negative one turns the
  // queries' signs, and with 0 the queries are multiplied by it instead)
  float factor = p.scale * (p.k_scale ? p.k_scale[kh] : 1.0f) * kLog2e;
  const bool turn = factor < 0.0f, zero = factor == 0.0f;
  factor = zero ? 1.0f : fabsf(factor);
  typename Mma<T>::op q[Steps];
  {
    const uint8_t* from = reinterpret_cast<const uint8_t*>(p.q + (s0 + member) * p.q_stride + (int64_t)(kh * p.group + head) * D);
#pragma unroll
    for (int s = 0; s < Steps; ++s) {
      uint32_t w[4];
      load_bytes<16>(from + 2 * S::q_dim(s, half_of), w);
      __builtin_memcpy(&q[s], w, 16);
    }
  }

  if (turn || zero) {
#pragma unroll
    for (int s = 0; s < Steps; ++s) {
      uint32_t w[4];
      __builtin_memcpy(w, &q[s], 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = zero ? not_finite_halves<T>(w[i]) : w[i] ^ 0x80008000u;
      __builtin_memcpy(&q[s], w, 16);
    }
  }
  f32x16 acc[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) acc[i] = zeros();
  // maximum and sum of the row; over: what the exponent of a score gets added
  float m = -FLT_MAX, l = 0.0f, over = FLT_MAX;
  bool infinite = false;  // a value that is not finite was taken out

  // (the accumulators stay where the matrix operations have them: without
  // this the rare branch that rescales them makes the compiler move them all
  // to other registers and back for every tile)
  auto in_place = [&]() __attribute__((always_inline)) {
    if (S::Waves > 4) return;
#pragma unroll
    for (int i = 0; i < PL; ++i) asm("" : "+a"(acc[i]));
#pragma unroll
    for (int i = 0; i < Steps; ++i) asm("" : "+a"(q[i]));
  };
  // --- a tile's operands, from LDS
  uint32_t k[D * TL::ES / 8];  // its keys
  typename Mma<V>::op v[2][PL];
  uint32_t bytes[TL::ES == 1 ? 2 : 1][TL::ES == 1 ? PL : 1][2];  // 8-bit values as they are read
  auto load_keys = [&](int step, int sub) __attribute__((always_inline)) {
    const uint8_t* row = lds + (step & 1) * kBuf + sub * S::TileBytes + r * Row;
#pragma unroll
    for (int i = 0; i < S::Pieces / 2; ++i) load_bytes<16>(row + 16 * ((2 * i + half_of) ^ S::mix_k(r)), &k[4 * i]);
  };
  auto key_op = [&](int s) __attribute__((always_inline)) {
    uint32_t w[4];
    if constexpr (TL::ES == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = k[4 * s + i];
    } else {
      Mma<T>::widen(k[2 * s], w);
      Mma<T>::widen(k[2 * s + 1], w + 2);
    }
    typename Mma<T>::op x;
    __builtin_memcpy(&x, w, 16);
    return x;
  };
  // operand (j, i) of the values is 32 dimensions of 16 of the tile's tokens:
  // a read that transposes gives lane l of 16 dimension l of the four tokens
  // (8-bit: eight) whose rows the 16 lanes name.  (Tokens 8 and 16 apart are
  // mixed alike.)
  const int side = lane >> 4 & 1, l16 = lane & 15;  // which 16 of the dimensions
  auto load_values = [&](int step, int sub) __attribute__((always_inline)) {
    const uint8_t* values = lds + (step & 1) * kBuf + kKeys + sub * S::TileBytes;
    if constexpr (TL::ES == 2) {
      const int t = 4 * half_of + (l16 >> 2);
      const uint8_t* row = values + t * Row + 8 * (l16 & 1);
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int at = 16 * ((4 * i + 2 * side + (l16 >> 1 & 1)) ^ S::mix_v(t));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const s16x4 four =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(row + at + (16 * j + 8 * x) * Row));
            __builtin_memcpy((uint8_t*)&v[j][i] + 8 * x, &four, 8);
          }
      }
    } else {
      const int t = 8 * (l16 >> 3) + 4 * half_of + (l16 >> 1 & 3);
      const uint8_t* row = values + t * Row + 8 * (l16 & 1);
#pragma unroll
      for (int i = 0; i < PL; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const i32x2 b = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (__attribute__((address_space(3))) i32x2*)(row + 16 * ((2 * i + side) ^ S::mix_v(t)) + 16 * j * Row));
          bytes[j][i][0] = b.x, bytes[j][i][1] = b.y;
        }
    }
  };
  auto widen_values = [&]() __attribute__((always_inline)) {
    if constexpr (TL::ES == 1) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          uint32_t w[4];
          Mma<V>::widen(bytes[j][i][0], w);
          Mma<V>::widen(bytes[j][i][1], w + 2);
          __builtin_memcpy(&v[j][i], w, 16);
        }
    }
  };

  // Step i of the workgroup: the tiles that buffer i % 2 holds, each wave its
  // stream's.  A wave reads a tile's operands while it works on the one
  // before, so when all have come to their last tile of a step its buffer is
  // free for the step after the next, and that step's loads have a step's
  // time to land.
  if (steps > 0) landed_barrier<0>();
  if (fetches && steps > 1) fetch(1);
  auto pages_of = [&](int step) __attribute__((always_inline)) {
    uint64_t v = 0;
    __builtin_memcpy(&v, has_page[step & 1], 2 * Subs);
    return (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)v) |
           (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32;
  };
  if (__all(none)) {
    // no row of this wave sees anything: it only fetches, and leaves its SIMD
    // to the other wave (256 sequences in two groups, a sixth of the row waves
    // empty: 44.0 -> 43.4 us)
#pragma unroll 1
    for (int step = 0; step + 1 < steps; ++step) {
      landed_barrier<0>();
      if (step + 2 < steps && fetches) {
        if (((step + 2) & 63) == 0) load_pages(step + 2);
        fetch(step + 2);
      }
    }
  } else if (it.tile + stream < it.tile_end) {
    uint64_t pages = pages_of(0);
    int step = 0, sub = stream;
    load_keys(0, sub);
#pragma unroll 1
    for (;;) {
      const int tile = it.tile + step * Subs + sub, t0 = tile * kTokens;
      load_values(step, sub);
      in_place();
      f32x16 s = zeros();
#pragma unroll
      for (int st = 0; st < Steps; ++st) s = mul32(key_op(st), q[st], s);
      widen_values();
      const uint32_t have = (uint32_t)(pages >> (16 * sub) & 1) | (uint32_t)(pages >> (16 * sub + 7) & 2);
      if (!(t0 >= lo_max && t0 <= hi_min - kTokens && have == 3)) {
        // some row does not see some token: no score there.  Nobody sees a
        // token outside lo_all .. hi_all - 1 or without a page; the values
        // of the others stay, but for those that would be NaN times a
        // probability of 0 (the rows that see them get them at the end)
        uint32_t is = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int t = t0 + 8 * (e >> 2) + 4 * half_of + (e & 3);
          if ((have >> (e >> 3) & 1) && t >= lo_all && t < hi_all) is |= 1u << e;
          s[e] = (is >> e & 1) && t >= lo && t < hi ? s[e] : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < PL; ++i) {
            uint32_t w[4];
            __builtin_memcpy(w, &v[j][i], 16);
#pragma unroll
            for (int n = 0; n < 4; ++n) {  // (tokens of scores 8 j + 2 n and the next)
              const uint32_t bits = is >> (8 * j + 2 * n);
              w[n] = finite_halves<V>(w[n] & ((bits & 1 ? 0xFFFFu : 0u) | (bits & 2 ? 0xFFFF0000u : 0u)), infinite);
            }
            __builtin_memcpy(&v[j][i], w, 16);
          }
      }
      // exponents of the probabilities (2^lift times them).  The maxima are
      // taken of these, whose products the compiler need not quieten first.
      float x[16];
      auto exponents = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = fmaf(s[i], factor, over);
      };
      exponents();
      float top = x[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
      if (__any(top > kSlack + Mma<V>::lift)) {
        float most = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) most = fmaxf(most, s[i]);
        const float mn = fmaxf(m, row_max(most) * factor);
        const float f = __builtin_amdgcn_exp2f(m - mn);
        l *= f;
#pragma unroll
        for (int i = 0; i < PL; ++i) acc[i] *= f;
        m = mn;
        over = Mma<V>::lift - mn;
        exponents();
      }
      // the next tile (after the last one, this one again)
      int next_step = step, next_sub = sub + streams;
      if (next_sub >= Subs) {
        next_step = step + 1, next_sub = stream;
        if (next_step < steps) {
          landed_barrier<0>();
          if (step + 2 < steps && fetches) {
            if (((step + 2) & 63) == 0) load_pages(step + 2);
            fetch(step + 2);
          }
          pages = pages_of(next_step);
        }
      }
      const bool done = next_step == steps || it.tile + next_step * Subs + next_sub >= it.tile_end;
      if (done) next_step = step, next_sub = sub;
      in_place();
      load_keys(next_step, next_sub);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_amdgcn_exp2f(x[8 * j + i]);
          l += e[i];
        }
        float rest[8];
        const typename Mma<V>::op hi = Mma<V>::split(e, rest), lo = Mma<V>::round(rest);
#pragma unroll
        for (int i = 0; i < PL; ++i) acc[i] = mul32(v[j][i], hi, acc[i]);
#pragma unroll
        for (int i = 0; i < PL; ++i) acc[i] = mul32(v[j][i], lo, acc[i]);
      }
      if (done) break;
      step = next_step, sub = next_sub;
    }
  }

  // the parts of the waves with the same rows into the chunk's: each brings
  // its sums to the largest maximum, then they are added up
  float(*const red)[RowF] = reinterpret_cast<float(*)[RowF]>(lds);  // [Waves * Rows]
  __syncthreads();  // (the tiles are read)
  l = none ? 0.0f : row_sum(l);
  m = none ? -FLT_MAX : m;
  if (half_of == 0) red_m[wave * S::Rows + r] = m;
  __syncthreads();
  {
    float mw = m;
    for (int w = wave & (row_waves - 1); w < Waves; w += row_waves) mw = fmaxf(mw, red_m[w * S::Rows + r]);
    const float f = none ? 0.0f : __builtin_amdgcn_exp2f(m - mw);
    float* const row = red[wave * S::Rows + r];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PL; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        f32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = none ? 0.0f : acc[i][4 * n + k] * f;
        nan |= any_nan(o);
        *reinterpret_cast<f32x4*>(row + 32 * i + 8 * n + 4 * half_of) = o;
      }
    if (half_of == 0) row[D] = mw, row[D + 1] = none ? 0.0f : l * f;
    infinite |= nan && l == l;
  }
  // Where an infinite or NaN value is in play: the sums of such values over the
  // item's tokens, which all threads form once (their order does not matter); a
  // row that sees only a part of these tokens forms its own (one infinite value
  // among 32768 tokens of 64 sequences: a call of 137 us, without one 109; with a
  // sum for every row 5.1 ms).
  const int all_from = max(lo_all, first_token(it.tile)), all_to = min(hi_all, first_token(it.tile_end));
  auto special_of = [&](int from, int to, int d) {
    return infinite_values<C, D>(table, reinterpret_cast<const typename C::bits_t*>(p.v_cache), p.pages, p.kv_heads, kh,
                                 p.page_shift, from, to, d);
  };
  infinite = __syncthreads_or(infinite);
  if (__builtin_expect(infinite, false)) {
    constexpr int kSlices = kThreads / (D / 4);
    if (threadIdx.x < D) special[threadIdx.x] = 0.0f;
    __syncthreads();
    const int d = 4 * (threadIdx.x % (D / 4)), slice = threadIdx.x / (D / 4);
    const uint32_t all = (uint32_t)max(all_to - all_from, 0), span = all / kSlices + 1;  // (tokens up to 2^31 - 16)
    const uint32_t from = min(all, slice * span), to = min(all, from + span);
    if (slice < kSlices && from < to) {
      const f32x4 y = special_of(all_from + (int)from, all_from + (int)to, d);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (y[j] != 0.0f) atomicAdd(&special[d + j], y[j]);
    }
    __syncthreads();
  }
  const int first_row = it.block * row_waves * S::Rows;
  float* const parts = p.prefix_parts + ((int64_t)it.row + ((int64_t)it.chunk * p.kv_heads + kh) * rows + first_row) * RowF;
#pragma unroll 1
  for (int i = threadIdx.x; i < row_waves * S::Rows * (D / 4); i += kThreads) {
    const int k = i / (D / 4), d = 4 * (i % (D / 4));
    if (first_row + k >= rows) break;
    f32x4 o = *reinterpret_cast<const f32x4*>(&red[k][d]);
    float sum = red[k][D + 1];
    for (int w = row_waves; w < Waves; w += row_waves) {
      o += *reinterpret_cast<const f32x4*>(&red[w * S::Rows + k][d]);
      sum += red[w * S::Rows + k][D + 1];
    }
    if (__builtin_expect(infinite, false) && sum == sum) {
      int from, to;
      visible(p, s0 + (first_row + k) / p.group, from, to);
      from = max(from, first_token(it.tile));
      to = min(min(to, prefix), first_token(it.tile_end));
      if (from < to) {
        f32x4 y = *reinterpret_cast<const f32x4*>(special + d);
        if (from != all_from || to != all_to) y = special_of(from, to, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = y[j] != 0.0f ? y[j] : o[j];
      }
    }
    *reinterpret_cast<f32x4*>(parts + (int64_t)k * RowF + d) = o;
    if (d == 0) *reinterpret_cast<float2*>(parts + (int64_t)k * RowF + D) = make_float2(red[k][D], sum);
  }
}

template <class T, class C>
void launch_dim(const AttnParams& p, int64_t head_dim, hipStream_t s) {
  auto grid = [&](int64_t least_rows) {
    // the plan, about prefix_target workgroups, and one more per key head and
    // row block
    return dim3((unsigned)(1 + p.prefix_target + p.kv_heads * ((int64_t)p.batch * p.group / least_rows + p.groups)));
  };
  switch (head_dim) {
#define BGG_PREFIX(D)                                                                                          \
  case D:                                                                                                      \
    hipLaunchKernelGGL((k_shared_prefix<T, C, D>),                                                             \
                       grid(PrefixShape<T, C, D>::Rows * PrefixShape<T, C, D>::Least),                  \
                       dim3(64 * PrefixShape<T, C, D>::Waves), 0, s, p);                                       \
    break
    BGG_PREFIX(64);
    BGG_PREFIX(96);
    BGG_PREFIX(128);
    BGG_PREFIX(192);
    BGG_PREFIX(256);
#undef BGG_PREFIX
  }
}

}  // namespace

namespace bgg {

int64_t prefix_part_floats(const bgg_cache_desc* c, int64_t q_heads, int64_t batch, int64_t target) {
  // an item has at most 256 rows (128 of wide heads) and there are target of
  // them, and each row one part more
  const int64_t D = c->head_dim;
  return (target * (D <= 128 ? 256 : 128) + batch * q_heads) * (D + 4);
}

void launch_prefix(const AttnParams& p, int32_t type, bool e4m3, int64_t head_dim, hipStream_t s) {
  if (type == BGG_TYPE_F16) {
    if (e4m3)
      launch_dim<F16, E4M3>(p, head_dim, s);
    else
      launch_dim<F16, F16>(p, head_dim, s);
  } else {
    if (e4m3)
      launch_dim<BF16, E4M3>(p, head_dim, s);
    else
      launch_dim<BF16, BF16>(p, head_dim, s);
  }
}

}  // namespace bgg
