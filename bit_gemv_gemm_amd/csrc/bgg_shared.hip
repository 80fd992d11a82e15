// The shared part of bgg_shared_attention: groups of sequences whose first
// pages are the same read those pages once.  With the members' query heads of
// a key head as rows, it is a product of many rows with the prefix, so it is
// bound by the matrix and vector units instead of the cache's bytes as soon
// as a group has more than a few members.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bgg_paged.h"
#include "bgg_shared.h"

using namespace bgg;

namespace {

constexpr int kThreads = 64 * kWaves;
constexpr int kGroupsMax = (int)kMaxBatch;

// Sum over the lanes up to and including this one, of larger of the two.
template <int MOVE, int ROWS>
__device__ __forceinline__ int max_from(int v) {
  return max(v, __builtin_amdgcn_update_dpp(0, v, MOVE, ROWS, 0xF, false));
}

// The groups, in LDS: group g has the sequences start[g] .. start[g + 1] - 1,
// `tokens` tokens of prefix, of which its sequences see lo .. hi - 1.
struct Groups {
  int start[kGroupsMax + 1], tokens[kGroupsMax], lo[kGroupsMax], hi[kGroupsMax];
};

// Largest g <= G - 1 with start[g] <= b (start[0] <= b).
__device__ __forceinline__ int group_of(const Groups& s, int G, int b) {
  int lo = 0, n = G;
#pragma unroll 1
  while (n > 1) {
    const int half = n >> 1;
    const bool right = s.start[lo + half] <= b;
    lo = right ? lo + half : lo;
    n = right ? n - half : half;
  }
  return lo;
}

__device__ __forceinline__ void read_groups(const AttnParams& p, Groups& s) {
  const int tid = threadIdx.x, G = p.groups;
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
      if (g <= G) s.start[g] = v;
      before = __builtin_amdgcn_readlane(v, 63);
    }
  }
  __syncthreads();
  for (int g = tid; g < G; g += kThreads) {
    const int b = s.start[g];
    const int pages = s.start[g + 1] > b ? p.shared_pages[b] : 0;
    s.tokens[g] = min(max(pages, 0), p.max_tokens >> p.page_shift) << p.page_shift;
    s.lo[g] = 0x7FFFFFFF;
    s.hi[g] = 0;
  }
  __syncthreads();
  for (int b = s.start[0] + tid; b < s.start[G]; b += kThreads) {
    int lo, n;
    visible(p, b, lo, n);
    const int g = group_of(s, G, b);
    n = min(n, s.tokens[g]);
    if (lo < n) {
      atomicMin(&s.lo[g], lo);
      atomicMax(&s.hi[g], n);
    }
  }
  __syncthreads();
}

// Chunks of a group's prefix, as even as the even size allows.
constexpr int kMinTiles = kWaves;
__device__ __forceinline__ int prefix_chunks(int tiles, int size) {
  return (tiles + size - 1) / size;
}

struct PrefixItem {
  int group, kh, block, chunk, chunks, row;  // row: the group's first row of the parts
  int tile, tile_end;
};

// The item of this workgroup; in `base` and `count`, if given, the first row
// and the chunks of every group.  Every wave works it out by itself.
template <int RB>
__device__ __forceinline__ bool find_prefix(const AttnParams& p, const Groups& s, int index, PrefixItem& it, int* base,
                                            int* count) {
  const int lane = threadIdx.x & 63, G = p.groups;
  const int per = (G + 63) / 64, g0 = min(G, lane * per), g1 = min(G, g0 + per);
  auto shape = [&](int g, int& tiles, int& blocks, int& rows) {
    tiles = tiles_of(s.lo[g], s.hi[g]);
    rows = (s.start[g + 1] - s.start[g]) * p.group;
    blocks = (rows + RB - 1) / RB;
  };
  float work = 0.0f;
  int tiles, blocks, rows;
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    shape(g, tiles, blocks, rows);
    work += (float)tiles * (float)blocks;
  }
  const float even = fminf(ceilf(wave_add(work) * (float)p.kv_heads / (float)p.prefix_target * 1.0001f), 1e8f);
  int size = 0, mine = 0, upto = 0;
#pragma unroll 1
  for (int k = 8; k <= 16; k += 2) {
    size = max(kMinTiles, (int)(even * (float)k * 0.125f));
    mine = 0;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      shape(g, tiles, blocks, rows);
      mine += prefix_chunks(tiles, size) * blocks;
    }
    upto = scan_add(mine);
    if (__builtin_amdgcn_readlane(upto, 63) * p.kv_heads <= p.prefix_target) break;
  }
  size = __builtin_amdgcn_readfirstlane(size);
  // rows of the parts before this lane's groups
  int lane_rows = 0;
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    shape(g, tiles, blocks, rows);
    lane_rows += prefix_chunks(tiles, size) * p.kv_heads * rows;
  }
  int row = scan_add(lane_rows) - lane_rows;
  if (base && threadIdx.x < 64) {
    int r = row;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      shape(g, tiles, blocks, rows);
      base[g] = r;
      count[g] = prefix_chunks(tiles, size);
      r += count[g] * p.kv_heads * rows;
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
#pragma unroll 1
  for (;; ++g) {
    shape(g, tiles, blocks, rows);
    const int n = prefix_chunks(tiles, size) * blocks;
    if (at < first + n) break;
    first += n;
    row += prefix_chunks(tiles, size) * p.kv_heads * rows;
  }
  it.group = __builtin_amdgcn_readfirstlane(g);
  it.kh = index % p.kv_heads;
  it.row = __builtin_amdgcn_readfirstlane(row);
  it.chunks = __builtin_amdgcn_readfirstlane(prefix_chunks(tiles, size));
  const int local = at - first;
  it.block = __builtin_amdgcn_readfirstlane(local % blocks);
  it.chunk = __builtin_amdgcn_readfirstlane(local / blocks);
  const int t0 = s.lo[g] / kTokens, each = (tiles + it.chunks - 1) / it.chunks;
  it.tile = __builtin_amdgcn_readfirstlane(t0 + it.chunk * each);
  it.tile_end = __builtin_amdgcn_readfirstlane(t0 + min(tiles, (it.chunk + 1) * each));
  return true;
}

// The schedule of the sequences' own tokens (one workgroup): bgg_attention's
// chunks, an entry each.
__device__ __forceinline__ void plan_own(const AttnParams& p, const Groups& s, const int* base, const int* count,
                                         int* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int H = p.kv_heads * p.head_blocks, G = p.groups;
  const int per = (p.batch + kThreads - 1) / kThreads, b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  auto own = [&](int b, int& lo, int& n) {
    visible(p, b, lo, n);
    const int g = group_of(s, G, b);
    SharedSeq q{0, 0, 0, 0};
    if (s.start[g] <= b && b < s.start[g + 1]) {
      q.tokens = s.tokens[g];
      q.chunks = count[g];
      q.rows = (s.start[g + 1] - s.start[g]) * p.group;
      q.row = base[g] + (b - s.start[g]) * p.group;
    }
    lo = max(lo, q.tokens);
    return q;
  };
  float* const sums = reinterpret_cast<float*>(scratch);
  float tiles = 0.0f;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    int lo, n;
    p.seqs[b] = own(b, lo, n);
    tiles += (float)tiles_of(lo, n);
  }
  tiles = wave_add(tiles);
  if (lane == 0) sums[wave] = tiles;
  __syncthreads();
  float all = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) all += sums[w];
  __syncthreads();
  const float even = fminf(ceilf(all * (float)H / (float)p.target_items * 1.0001f), 1e8f);
  int size = 0, mine = 0, before = 0;
#pragma unroll 1
  for (int k = 8; k <= 16; k += 2) {
    size = max(1, (int)(even * (float)k * 0.125f));
    mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      int lo, n;
      own(b, lo, n);
      mine += both_counts(chunks_of(tiles_of(lo, n), size));
    }
    const int upto = scan_add(mine);
    if (lane == 63) scratch[wave] = upto;
    __syncthreads();
    before = upto - mine;
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) before += scratch[w];
      total += scratch[w];
    }
    __syncthreads();
    if (tid == 0) *p.own_count = total & 0xFFFF;
    if (p.batch * H > p.target_items || (total & 0xFFFF) * H <= p.target_items) break;
  }
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    OwnItem it;
    own(b, it.lo, it.n);
    const int t = tiles_of(it.lo, it.n), first = it.lo / kTokens, chunks = chunks_of(t, size);
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
template <class C>
__device__ __forceinline__ uint32_t without_infinite(uint32_t w, bool& found) {
  if constexpr (sizeof(typename C::bits_t) == 2) {
    constexpr uint32_t e = (uint32_t)C::exponent;
    const bool lo = (w & e) == e, hi = (w & (e << 16)) == (e << 16);
    found |= lo | hi;
    return (lo ? 0u : w & 0xFFFFu) | (hi ? 0u : w & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool bad = ((w >> (8 * i)) & 0x7Fu) == 0x7Fu;
      found |= bad;
      w = bad ? w & ~(0xFFu << (8 * i)) : w;
    }
    return w;
  }
}

template <class T, class C, int D>
struct PrefixShape {
  // blocks of 16 rows that a wave keeps in registers (queries, accumulators)
  static constexpr int Blocks = D <= 128 ? 4 : 2;
  static constexpr int Rows = 16 * Blocks;
  static constexpr int RowF = D + 4;  // floats of a row of the parts: values, maximum, sum
};

template <class T, class C, int D>
__global__ void __launch_bounds__(kThreads, 1) k_shared_prefix(AttnParams p) {
  using TL = Tile<T, C, D>;
  using V = typename TL::V;
  using S = PrefixShape<T, C, D>;
  constexpr int PL = TL::PL, NB = S::Blocks, RowF = S::RowF;
  __shared__ union {
    struct {
      Groups groups;
      int base[kGroupsMax], count[kGroupsMax], scratch[kWaves];
    } plan;
    __attribute__((aligned(16))) float red[kWaves][kHeads][RowF];
  } lds;
  __shared__ float red_m[kWaves][kHeads], red_l[kWaves][kHeads];

  read_groups(p, lds.plan.groups);
  PrefixItem it;
  if (blockIdx.x == 0) {
    find_prefix<S::Rows>(p, lds.plan.groups, 0, it, lds.plan.base, lds.plan.count);
    __syncthreads();
    plan_own(p, lds.plan.groups, lds.plan.base, lds.plan.count, lds.plan.scratch);
    return;
  }
  if (!find_prefix<S::Rows>(p, lds.plan.groups, blockIdx.x - 1, it, nullptr, nullptr)) return;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kh = it.kh;
  const int s0 = lds.plan.groups.start[it.group], rows = (lds.plan.groups.start[it.group + 1] - s0) * p.group;
  const int prefix = lds.plan.groups.tokens[it.group];
  const int lo_all = lds.plan.groups.lo[it.group], hi_all = lds.plan.groups.hi[it.group];

  // the lane's row of each block: queries and the tokens it sees
  float factor = p.scale * (p.k_scale ? p.k_scale[kh] : 1.0f) * kLog2e;
  typename Mma<T>::op q[NB][TL::Steps];
  int lo[NB], hi[NB];
  int lo_max = 0, hi_min = 0x7FFFFFFF;
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const int row = it.block * S::Rows + 16 * c + r;
    const int member = row / p.group, b = s0 + min(member, rows / p.group - 1);
    lo[c] = 0, hi[c] = 0x7FFFFFFF;
    if (row < rows) {
      visible(p, b, lo[c], hi[c]);
      hi[c] = min(hi[c], prefix);
      lo_max = max(lo_max, lo[c]);
      hi_min = min(hi_min, hi[c]);
    }
#pragma unroll
    for (int s = 0; s < TL::Steps; ++s) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (row < rows)
        load_bytes<16>(reinterpret_cast<const uint8_t*>(p.q + b * p.q_stride +
                                                        (int64_t)(kh * p.group + row - member * p.group) * D + TL::q_dim(s, g)),
                       w);
      __builtin_memcpy(&q[c][s], w, 16);
    }
  }
  // over the rows (the same in each of the four lanes of a row)
#pragma unroll
  for (int s = 1; s < 16; s <<= 1) {
    lo_max = max(lo_max, __shfl_xor(lo_max, s));
    hi_min = min(hi_min, __shfl_xor(hi_min, s));
  }
  lo_max = __builtin_amdgcn_readfirstlane(lo_max);
  hi_min = __builtin_amdgcn_readfirstlane(hi_min);
  __syncthreads();  // (the plan is read: its place takes the sums)

  f32x4 acc[NB][PL];
  float m[NB], l[NB];
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    m[c] = -FLT_MAX, l[c] = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; ++i) acc[c][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  bool infinite = false;  // a value that is not finite was taken out

  // the page numbers of this wave's tiles, a tile per lane (64 at a time)
  const int32_t* table = p.table + s0 * p.table_stride;
  int page_of[2] = {-1, -1};
  auto load_pages = [&](int tile) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = (tile + kWaves * lane) * kTokens + 16 * j;
      page_of[j] = tile + kWaves * lane < it.tile_end && t < hi_all ? table[t >> p.page_shift] : -1;
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
    __builtin_amdgcn_sched_barrier(0);
    tl.load_v(now.v, lane);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int tile = first, step = 0; tile < it.tile_end; tile += kWaves, ++step) {
    const bool more = tile + kWaves < it.tile_end;
    f32x4 s[NB][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int c = 0; c < NB; ++c) s[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < TL::Steps; ++st) {
        const typename Mma<T>::op k = tl.k_op(j, st);
#pragma unroll
        for (int c = 0; c < NB; ++c) s[c][j] = Mma<T>::mul(k, q[c][st], s[c][j]);
      }
    }
    if (more && ((step + 1) & 63) == 0) load_pages(tile + kWaves);
    const Place next = place(step + more, tile + (more ? kWaves : 0));
    __builtin_amdgcn_sched_barrier(0);
    tl.load_k(next.k, lane);
    __builtin_amdgcn_sched_barrier(0);
    const int t0 = tile * kTokens;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[c][e >> 2][e & 3] *= factor;
    if (!(t0 >= lo_max && t0 + kTokens <= hi_min && now.ok[0] && now.ok[1])) {
      // some row does not see some token: no score there.  Nobody sees a
      // token outside lo_all .. hi_all - 1 or without a page; the values of
      // the others stay, but for those that would be NaN times a probability
      // of 0 (the rows that see them get them at the end)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = t0 + 16 * (e >> 2) + 4 * g + (e & 3);
        const bool is = now.ok[e >> 2] && t >= lo_all && t < hi_all;
#pragma unroll
        for (int w = 0; w < TL::W0 + TL::W1; ++w) {
          tl.v[e][w] = is ? tl.v[e][w] : 0u;
          tl.v[e][w] = without_infinite<C>(tl.v[e][w], infinite);
        }
#pragma unroll
        for (int c = 0; c < NB; ++c)
          s[c][e >> 2][e & 3] = is && t >= lo[c] && t < hi[c] ? s[c][e >> 2][e & 3] : -INFINITY;
      }
    }
    float top[NB];
    bool raise = false;
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      top[c] = fmaxf(fmaxf(fmaxf(s[c][0][0], s[c][0][1]), fmaxf(s[c][0][2], s[c][0][3])),
                     fmaxf(fmaxf(s[c][1][0], s[c][1][1]), fmaxf(s[c][1][2], s[c][1][3])));
      raise |= top[c] > m[c] + kSlack;
    }
    if (__any(raise)) {
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        const float mn = fmaxf(m[c], column_max(top[c]));
        const float f = __builtin_amdgcn_exp2f(m[c] - mn);
        l[c] *= f;
#pragma unroll
        for (int i = 0; i < PL; ++i) acc[c][i] *= f;
        m[c] = mn;
      }
    }
    typename Mma<V>::op pr[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(s[c][i >> 2][i & 3] - m[c] + Mma<V>::lift);
        l[c] += e[i];
      }
      pr[c] = Mma<V>::round(e);
    }
#pragma unroll
    for (int i = 0; i < PL; i += 2) {
      typename Mma<V>::op a, b;
      tl.v_ops(i, a, b);
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        acc[c][i] = Mma<V>::mul(a, pr[c], acc[c][i]);
        acc[c][i + 1] = Mma<V>::mul(b, pr[c], acc[c][i + 1]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    tl.load_v(next.v, lane);
    __builtin_amdgcn_sched_barrier(0);
    now = next;
  }

  // the waves' parts, a block after the other, into the chunk's
  infinite = __syncthreads_or(infinite);
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const float sum = column_sum(l[c]);
    if (c) __syncthreads();  // (the block before is read)
    if (g == 0) red_m[wave][r] = m[c], red_l[wave][r] = sum;
    __syncthreads();
    float mw = red_m[0][r];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mw = fmaxf(mw, red_m[w][r]);
    const float f = __builtin_amdgcn_exp2f(m[c] - mw);
#pragma unroll
    for (int i = 0; i < PL; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) lds.red[wave][r][TL::dim(4 * g + k, i)] = acc[c][i][k] * f;
    __syncthreads();
    for (int i = threadIdx.x; i < kHeads * (D / 4); i += kThreads) {
      const int h = i / (D / 4), d = 4 * (i % (D / 4)), row = it.block * S::Rows + 16 * c + h;
      if (row >= rows) break;
      float mh = red_m[0][h], lh = 0.0f;
      f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 1; w < kWaves; ++w) mh = fmaxf(mh, red_m[w][h]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        lh += red_l[w][h] * __builtin_amdgcn_exp2f(red_m[w][h] - mh);
        o += *reinterpret_cast<const f32x4*>(&lds.red[w][h][d]);
      }
      if (__builtin_expect(infinite || any_nan(o), false) && lh == lh) {
        int seen_lo, seen_hi;
        visible(p, s0 + row / p.group, seen_lo, seen_hi);
        seen_lo = max(seen_lo, it.tile * kTokens);
        seen_hi = min(min(seen_hi, prefix), it.tile_end * kTokens);
        if (seen_lo < seen_hi) {
          const f32x4 x = infinite_values<C, D>(table, reinterpret_cast<const typename C::bits_t*>(p.v_cache), p.pages,
                                                p.kv_heads, kh, p.page_shift, seen_lo, seen_hi, d);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = x[k] != 0.0f ? x[k] : o[k];
        }
      }
      float* out = p.prefix_parts + ((int64_t)it.row + ((int64_t)it.chunk * p.kv_heads + kh) * rows + row) * RowF;
      *reinterpret_cast<f32x4*>(out + d) = o;
      if (d == 0) *reinterpret_cast<float2*>(out + D) = make_float2(mh, lh);
    }
  }
}

template <class T, class C>
void launch_dim(const AttnParams& p, int64_t head_dim, hipStream_t s) {
  const dim3 block(kThreads);
  auto grid = [&](int64_t rows_of_block) {
    // the plan, about prefix_target workgroups, and one more per key head and
    // row block
    return dim3((unsigned)(1 + p.prefix_target + p.kv_heads * ((int64_t)p.batch * p.group / rows_of_block + p.groups)));
  };
  switch (head_dim) {
#define BGG_PREFIX(D) \
  case D: hipLaunchKernelGGL((k_shared_prefix<T, C, D>), grid(PrefixShape<T, C, D>::Rows), block, 0, s, p); break
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
  const int64_t D = c->head_dim;
  return (target * (D <= 128 ? 64 : 32) + batch * q_heads) * (D + 4);
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
