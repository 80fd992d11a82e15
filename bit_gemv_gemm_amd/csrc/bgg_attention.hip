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
//
// bgg_shared_attention's second launch is the same kernel (SHARED): the
// sequences' own tokens, from a schedule that the first launch left, and at
// the end the parts of the prefix, added in the order of its chunks.  It is
// bound by the own tokens' bytes and the parts': 16 sequences of up to 2000
// own tokens of 4 x 256 bf16 19.6 us (61 MB), 256 of up to 200 of 8 x 128 bf16
// 19.1 us (105 MB, from the Infinity Cache, and 30 MB of parts).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bgg_shared.h"

using namespace bgg;

namespace {

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

// The parts of the prefix that sequence b shares (bgg_shared.hip), with the
// accumulator, maximum and sum of values d .. d + 3 of head i of key head kh.
template <int D>
__device__ __forceinline__ void add_prefix(const AttnParams& p, int b, int kh, int i, int d, f32x4& o, float& m,
                                           float& l) {
  constexpr int kFlight = 8, RowF = D + 4;  // (parts in flight: of 4, 8 and 16, 8 measured best)
  const SharedSeq q = p.seqs[b];
  const float* at = p.prefix_parts + ((int64_t)q.row + (int64_t)kh * q.rows + i) * RowF;
  const int64_t step = (int64_t)p.kv_heads * q.rows * RowF;
  const f32x4 own = o;
#pragma unroll 1
  for (int c0 = 0; c0 < q.chunks; c0 += kFlight) {
    f32x4 x[kFlight];
    float2 ml[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const float* row = at + min(c0 + j, q.chunks - 1) * step;
      x[j] = *reinterpret_cast<const f32x4*>(row + d);
      ml[j] = *reinterpret_cast<const float2*>(row + D);
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) mn = fmaxf(mn, ml[j].x);
    const float f = __builtin_amdgcn_exp2f(m - mn);
    o *= f;
    l *= f;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      // (a part past the last is left out by selects: its values may be infinite)
      const bool in = c0 + j < q.chunks;
      const float w = __builtin_amdgcn_exp2f(ml[j].x - mn);
      l = in ? fmaf(ml[j].y, w, l) : l;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = in ? fmaf(x[j][k], w, o[k]) : o[k];
    }
    m = mn;
  }
  if (__builtin_expect(__any(any_nan(o)), false) && any_nan(o) && l == l) {
    f32x4 s = {not_finite(own[0]), not_finite(own[1]), not_finite(own[2]), not_finite(own[3])};
#pragma unroll 1
    for (int c = 0; c < q.chunks; ++c) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(at + c * step + d);
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += not_finite(x[k]);
    }
    take_infinite(o, s);
  }
}

// The parts of a sequence's chunks (at parts, parts + step, ...) into its
// output: each chunk's weight 2^(m_c - m), then the weighted rows, four
// values (a column) per thread and step; with fewer columns than threads the
// threads also share the chunks out among them.  The maxima and sums and the
// first columns are loaded together, so that up to eight chunks cost one trip
// to memory.  This code runs once, by one workgroup per sequence and head
// block, so its instructions come from memory too: it is kept short by loops
// (unrolled to 16 parts in flight and three columns per thread it took 9 us
// for 32 chunks of 6 x 128).  `lds` holds 32 most_chunks floats.
template <class T, class V, int D, bool SHARED, int WAVES>
__device__ __forceinline__ void join_parts(const AttnParams& p, const Item& it, const float* parts,
                                           int64_t step, int rows, int heads, int h0, float vs,
                                           float* lds, float* lds16) {
  constexpr int kThreads = 64 * WAVES, kRows = kThreads / 16;  // threads of a head
  constexpr int kFlight = 8;                                    // a thread's parts in flight
  const int tid = threadIdx.x, hr = tid & 15, cr = tid >> 4;
  const int columns = heads * (D / 4);
  const int share = columns >= kThreads ? 1 : kThreads / columns;  // threads per column
  const int part_of = share > 1 ? tid / columns : 0;
  int col = share > 1 ? tid % columns : tid;
  float* weight = lds;                            // [chunks][16]
  float* sum = lds + 16 * most_chunks(WAVES);     // [chunks][16]

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
    float m = heads_m[h], l = heads_l[h];
    if constexpr (SHARED) {
      const int kh = it.head_block / p.head_blocks;
      add_prefix<D>(p, it.b, kh, h0 + h - kh * p.group, 4 * (col % (D / 4)), o, m, l);
    }
    store_out<T, V>(p, it.b, h0 + h, D, 4 * (col % (D / 4)), o, m, l, vs);
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
// arrives last adds the parts in chunk order.  SHARED: the items are
// bgg_shared.hip's, of the sequences' own tokens, and the parts of the prefix
// join at the end.
template <class T, class C, int D, bool SHARED, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, sizeof(typename C::bits_t) * D > 384 ? 1 : 2) k_paged_attention(AttnParams p) {
  using TL = Tile<T, C, D>;
  using V = typename TL::V;
  constexpr int PL = TL::PL;
  constexpr int RowF = D + 4;  // floats between heads in LDS
  // the waves' accumulators, then join_parts' weights and sums
  constexpr int kRed = WAVES * kHeads * RowF, kJoin = 32 * most_chunks(WAVES);
  __shared__ __attribute__((aligned(16))) float lds[kRed > kJoin ? kRed : kJoin];
  __shared__ float red_m[WAVES][kHeads], red_l[WAVES][kHeads], red_j[64 * WAVES + 32];
  static_assert(4 * 64 * WAVES <= 16 * most_chunks(WAVES), "the shares of the columns fit");
  float(*red)[kHeads][RowF] = reinterpret_cast<float(*)[kHeads][RowF]>(lds);
  __shared__ uint32_t arrived;

  Item it;
  if constexpr (SHARED) {
    const int H = p.kv_heads * p.head_blocks, at = blockIdx.x / H;
    if (at >= *p.own_count) return;
    const OwnItem e = p.own_items[at];
    it = Item{e.b, (int)blockIdx.x % H, e.chunk, e.chunks, e.part, e.lo, e.n, e.tile, e.tile_end};
  } else {
    if (!find_item(p, blockIdx.x, it)) return;
  }
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
      const int t = (tile + WAVES * lane) * kTokens + 16 * j;
      // (SHARED: an entry below it.lo may be one of the prefix, which is not this sequence's to read)
      const bool in = tile + WAVES * lane < it.tile_end && t < it.n && (!SHARED || t + 16 > it.lo);
      page_of[j] = in ? table[t >> p.page_shift] : -1;
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
  for (int tile = first, step = 0; tile < it.tile_end; tile += WAVES, ++step) {
    // the tile after this one, or this one again (loads without a branch
    // keep the waits for the loads before them exact)
    const bool more = tile + WAVES < it.tile_end;
    // scores of head r: tokens 16 j + 4 g + i
    f32x4 s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < TL::Steps; ++st) s[j] = Mma<T>::mul(tl.k_op(j, st), q[st], s[j]);
    }
    if (more && ((step + 1) & 63) == 0) load_pages(tile + WAVES);
    const Place next = place(step + more, tile + (more ? WAVES : 0));
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
  for (int w = 1; w < WAVES; ++w) mw = fmaxf(mw, red_m[w][r]);
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
  for (int i = threadIdx.x; i < columns; i += 64 * WAVES) {
    const int h = i / (D / 4), d = 4 * (i % (D / 4));
    float mh = red_m[0][h], lh = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 1; w < WAVES; ++w) mh = fmaxf(mh, red_m[w][h]);
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
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
      if constexpr (SHARED) add_prefix<D>(p, it.b, kh, hb * kHeads + h, d, o, mh, lh);
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
  join_parts<T, V, D, SHARED, WAVES>(p, it, part - (int64_t)it.chunk * H * slot, H * slot, rows, heads, h0, vs,
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
constexpr int64_t kSingle = 4;  // items of one wave that are cut in the place of one of four
static_assert(2 * kSingle * kMaxItems * 4 <= kCounterBytes, "a counter per part");

uint64_t own_part_bytes(const bgg_cache_desc* c, int64_t q_heads, int64_t parts) {
  return align256(4 * (uint64_t)(parts * part_floats(std::min<int64_t>(kHeads, q_heads / c->kv_heads), c->head_dim)));
}

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
  p.total_bytes = kCounterBytes + own_part_bytes(c, q_heads, p.parts);
  return p;
}

template <class T, class C, bool SHARED, int WAVES>
void launch_dim(const AttnParams& p, int64_t items, int64_t head_dim, hipStream_t s) {
  const dim3 grid((unsigned)items), block(64 * WAVES);
  switch (head_dim) {
    case 64: hipLaunchKernelGGL((k_paged_attention<T, C, 64, SHARED, WAVES>), grid, block, 0, s, p); break;
    case 96: hipLaunchKernelGGL((k_paged_attention<T, C, 96, SHARED, WAVES>), grid, block, 0, s, p); break;
    case 128: hipLaunchKernelGGL((k_paged_attention<T, C, 128, SHARED, WAVES>), grid, block, 0, s, p); break;
    case 192: hipLaunchKernelGGL((k_paged_attention<T, C, 192, SHARED, WAVES>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((k_paged_attention<T, C, 256, SHARED, WAVES>), grid, block, 0, s, p); break;
  }
}

template <bool SHARED, int WAVES>
void launch_attention(const AttnParams& p, int64_t items, int32_t type, bool e4m3, int64_t head_dim, hipStream_t s) {
  if (type == BGG_TYPE_F16) {
    if (e4m3)
      launch_dim<F16, E4M3, SHARED, WAVES>(p, items, head_dim, s);
    else
      launch_dim<F16, F16, SHARED, WAVES>(p, items, head_dim, s);
  } else {
    if (e4m3)
      launch_dim<BF16, E4M3, SHARED, WAVES>(p, items, head_dim, s);
    else
      launch_dim<BF16, BF16, SHARED, WAVES>(p, items, head_dim, s);
  }
}

// What bgg_shared_attention's workspace holds behind bgg_paged_attention's.
struct SharedPlan {
  uint64_t items, seqs, parts, total_bytes;  // byte offsets
};
SharedPlan plan_shared(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  SharedPlan p;
  // (kSingle times the items only if the batch alone is as many)
  const int64_t heads = c->kv_heads * ceil_div(q_heads / c->kv_heads, kHeads);
  const int64_t items = std::max<int64_t>(kMaxItems, std::min(kSingle * kMaxItems, batch * heads));
  p.items = kCounterBytes + own_part_bytes(c, q_heads, 2 * items) + 256;  // (the count before it)
  p.seqs = p.items + align256((items + batch) * sizeof(OwnItem));
  p.parts = p.seqs + align256(batch * sizeof(SharedSeq));
  p.total_bytes = p.parts + align256(4 * (uint64_t)prefix_part_floats(c, q_heads, batch, kMaxItems));
  return p;
}

bool sizes_ok(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  return check_cache(c) == BGG_OK && q_heads >= 1 && q_heads <= kMaxQHeads && q_heads % c->kv_heads == 0 && batch >= 1 &&
         batch <= kMaxBatch;
}

// The call, its arguments checked; shared: nullptr without groups.
bgg_status attend(const char* who, const bgg_cache_desc* c, const bgg_attention_args* a, const bgg_shared_args* shared,
                  void* stream) {
  if (a->batch == 0) return BGG_OK;
  const AttnPlan plan = plan_attention(c, a->q_heads, a->batch);
  const SharedPlan more = shared ? plan_shared(c, a->q_heads, a->batch) : SharedPlan{};
  const uint64_t need = shared ? more.total_bytes : plan.total_bytes;
  if (a->workspace_bytes < need)
    return fail(BGG_ERR_BUFFER, "%s: workspace has %zu bytes, needs %llu", who, a->workspace_bytes,
                (unsigned long long)need);
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
  const bool e4m3 = c->type == BGG_TYPE_E4M3;
  hipStream_t s = (hipStream_t)stream;
  if (!shared || shared->groups == 0) {
    launch_attention<false, kWaves>(p, plan.items, a->type, e4m3, c->head_dim, s);
    return hip_check(who);
  }
  uint8_t* const w = (uint8_t*)a->workspace;
  p.group_starts = shared->group_starts_dev;
  p.shared_pages = shared->shared_pages_dev;
  p.groups = (int)shared->groups;
  p.prefix_target = (int)plan.target;
  // A batch of so many sequences and head blocks fills the GPU with one wave
  // for each, and the starts and ends of workgroups of four cost more than
  // four waves to a sequence save; chunks are then cut for kSingle times as many
  // items.  One wave and four, us (8 key heads of 128 f16, 128, 256, 512 and 1024
  // sequences): up to 40 own tokens each 12.1, 17.0, 24.4, 39.4 and 14.1, 22.1, 35.0,
  // 64.1; up to 200 18.4, 28.6, 48.2, 106 and 21.4, 33.8, 59.3, 126; up to 1000
  // 70.6, 130, 232, 415 and 68.2, 131, 218, 404; up to 100 but for one of 65536 76.8,
  // 86.5, 104, 128 and 66.8, 79.2, 98.6, 135 (with chunks for as many items as four
  // waves have 84.4, 103, 122, 163).  Heads of 256 bf16 gain more (up to 200: 54.7
  // and 81.7), short 8-bit rows lose most behind one long sequence (128 of e4m3
  // heads of 64: 38.6 and 22.5).
  const bool single = a->batch * plan.heads >= kSingle * plan.target;
  p.own_target = (int)(single ? kSingle * plan.target : plan.target);
  p.own_chunks = most_chunks(single ? 1 : kWaves);
  p.own_count = (int32_t*)(w + more.items - 256);
  p.own_items = (OwnItem*)(w + more.items);
  p.seqs = (SharedSeq*)(w + more.seqs);
  p.prefix_parts = (float*)(w + more.parts);
  const int64_t items = p.own_target + a->batch * plan.heads;
  launch_prefix(p, a->type, e4m3, c->head_dim, s);
  const bgg_status st = hip_check(who);
  if (st) return st;
  if (!single)
    launch_attention<true, kWaves>(p, items, a->type, e4m3, c->head_dim, s);
  else
    launch_attention<true, 1>(p, items, a->type, e4m3, c->head_dim, s);
  return hip_check(who);
}

}  // namespace

extern "C" {

size_t bgg_attention_workspace_size(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  return sizes_ok(c, q_heads, batch) ? (size_t)plan_attention(c, q_heads, batch).total_bytes : 0;
}

bgg_status bgg_paged_attention(const bgg_cache_desc* c, const bgg_attention_args* a, void* stream) {
  const bgg_status st = check_attention(c, a);
  return st ? st : attend("bgg_paged_attention", c, a, nullptr, stream);
}

size_t bgg_shared_attention_workspace_size(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  return sizes_ok(c, q_heads, batch) ? (size_t)plan_shared(c, q_heads, batch).total_bytes : 0;
}

bgg_status bgg_shared_attention(const bgg_cache_desc* c, const bgg_attention_args* a, const bgg_shared_args* shared,
                                void* stream) {
  const bgg_status st = check_shared(c, a, shared);
  return st ? st : attend("bgg_shared_attention", c, a, shared, stream);
}

}  // extern "C"
