// Page tables and slots of a serving batch's step, from the lengths of its
// sequences and a stack of free pages: prefix sums over the sequences, then
// a position and a slot per row.
//
// k_cache_plan is one workgroup: pages given back, who is served, the new
// lengths (sums over up to 4096 sequences, in 32 bits: the call bounds what
// they add up to), and the rows of a small step.  A page given back or a row
// looks its sequence up in the sums (in LDS, by halving); a row takes its page
// from the table or, where the page is new, straight from the stack, so no row
// waits for another's entry of the table.  k_cache_fill writes the rows of a
// large step.  Both are bound by their chain of dependent steps (lengths, sums,
// table, slot) and by the time a launch takes: of one sequence 2.2 us, of 64
// with a token each 2.7 us.  4096 prompts of 1000000 rows, a tenth of the
// sequences ending: 7.4 us for the plan and 7.9 us for the 12 bytes written per
// row (2.4 us at the rate of a large copy).  What stays long is a step in which
// very many pages come back at once: about a microsecond per 4096 of them,
// since one workgroup orders them all.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bgg_cache.h"
#include "bgg_device.h"

using namespace bgg;

namespace {

struct AssignParams {
  const int32_t *lengths, *counts, *shared;
  int32_t* table;
  int64_t table_stride;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t *lengths_out, *free_count_out, *past, *starts, *positions;
  int64_t* slots;
  int batch, rows, width, capacity, pages, page_shift;
};

constexpr uint32_t kNotServed = 0xFFFFFFFFu;
constexpr int kEach = 4;  // rows of a thread of k_cache_fill
constexpr int kBack = 4;  // pages given back at a time by a thread

// What fill() needs of the sequences, in LDS.
template <int N>
struct Sums {
  uint32_t end[N];    // rows up to and with this sequence (at most T + 1)
  uint32_t taken[N];  // new pages before this sequence; kNotServed
  uint32_t past[N];
};

template <int MOVE, int ROWS>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, MOVE, ROWS, 0xF, false);
}
// Sums over the threads before this one, of two values at once, and the
// second's over all.  The first is cut to `most` in every step (cut sums add
// up to cut sums), so that it stays in 32 bits.
template <int THREADS>
__device__ __forceinline__ void sums_before(uint32_t& a, uint32_t& b, uint32_t& all_b, uint32_t most,
                                            uint32_t (*waves)[THREADS / 64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = a, y = b;
#define BGG_SCAN_STEP(MOVE, ROWS) \
  x = min(x + from_lane<MOVE, ROWS>(x), most), y += from_lane<MOVE, ROWS>(y)
  BGG_SCAN_STEP(0x111, 0xF);  // row_shr:1
  BGG_SCAN_STEP(0x112, 0xF);
  BGG_SCAN_STEP(0x114, 0xF);
  BGG_SCAN_STEP(0x118, 0xF);
  BGG_SCAN_STEP(0x142, 0xA);  // row_bcast:15 into rows 1, 3
  BGG_SCAN_STEP(0x143, 0xC);  // row_bcast:31 into rows 2, 3
#undef BGG_SCAN_STEP
  if (lane == 63) waves[0][wave] = x, waves[1][wave] = y;
  const uint32_t x_before = __shfl_up(x, 1);
  a = lane ? x_before : 0u;
  b = y - b;
  __syncthreads();
  all_b = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) a = min(a + waves[0][w], most), b += waves[1][w];
    all_b += waves[1][w];
  }
  __syncthreads();
}

// A barrier for what is in LDS: loads and stores of memory stay under way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// First i < n with v[i] > x (n if none).
__device__ __forceinline__ int first_above(const uint32_t* v, int n, uint32_t x) {
  int lo = 0;
#pragma unroll 1
  while (n > 0) {
    const int half = n >> 1;
    const bool right = v[lo + half] <= x;
    lo = right ? lo + half + 1 : lo;
    n = right ? n - half - 1 : half;
  }
  return lo;
}

// The page number of a row's token is read from the stack where its page is
// new (`fresh`), else from its entry of the table.
struct Row {
  int32_t position = 0, page = -1;
  int32_t* cell = nullptr;
  bool fresh = false;
};
// `i` counts the sequence's rows, `top` is the height of the stack before
// pages were taken.
__device__ __forceinline__ Row row_of(const AssignParams& p, int b, uint32_t i, uint32_t past, uint32_t taken, uint32_t top) {
  Row r;
  r.position = (int32_t)(past + i);
  const int entry = r.position >> p.page_shift, held = (int)((past + (1u << p.page_shift) - 1) >> p.page_shift);
  r.cell = p.table + b * p.table_stride + entry;
  r.fresh = entry >= held;
  r.page = *(r.fresh ? p.free_pages + (top - 1 - (taken + (uint32_t)(entry - held))) : r.cell);
  return r;
}
__device__ __forceinline__ int64_t slot_of(const AssignParams& p, const Row& r) {
  const int in_page = r.position & ((1 << p.page_shift) - 1);
  if (r.fresh && in_page == 0) *r.cell = r.page;  // (a new page's first token is always new)
  return r.page >= 0 && r.page < p.pages ? ((int64_t)r.page << p.page_shift) + in_page : -1;
}

// The step of a whole batch, or with FILL off all but its rows.
template <int THREADS, int PER, bool FILL>
__global__ void __launch_bounds__(THREADS) k_cache_plan(AssignParams p) {
  constexpr int N = THREADS * PER;
  __shared__ Sums<N> s;
  __shared__ uint32_t waves[2][THREADS / 64];
  __shared__ uint32_t last_taken;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t most = (uint32_t)p.rows + 1, cells = (1u << p.page_shift) - 1;
  const uint32_t all = (uint32_t)p.width << p.page_shift;  // (below 2^31)
  if (tid == 0) last_taken = 0;
  uint32_t top = (uint32_t)min(max(p.free_count[0], 0), p.capacity);

  uint32_t past[PER], count[PER], back[PER], rows = 0, backs = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    past[i] = count[i] = back[i] = 0;
    if (b < p.batch) {
      const int c = p.counts[b];
      const uint32_t n = min((uint32_t)max(p.lengths[b], 0), all);
      past[i] = n;
      if (c < 0) {
        const uint32_t low = p.shared ? (uint32_t)min(max(p.shared[b], 0), p.width) << p.page_shift : 0u;
        const uint32_t gone = 0u - (uint32_t)c;
        past[i] = min(n, max(gone < n ? n - gone : 0u, low));
        back[i] = ((n + cells) >> p.page_shift) - ((past[i] + cells) >> p.page_shift);
      } else {
        count[i] = (uint32_t)c;
      }
    }
    rows = min(rows + min(count[i], most), most);
    backs += back[i];
  }
  uint32_t row = rows, entry = backs, entries;
  sums_before<THREADS>(row, entry, entries, most, waves);

  // pages given back: all their table entries in one row, from its end
  if (entries) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      entry += back[i];
      s.end[tid * PER + i] = entry;
      s.past[tid * PER + i] = (past[i] + cells) >> p.page_shift;  // first entry given back
    }
    __syncthreads();
    // (kBack neighbours per thread, loaded together and a round ahead: one at a
    // time, 4096 sequences took 16.1 us in all, not 7.4)
    int32_t page[kBack], next[kBack];
    auto load_entries = [&](int32_t(&v)[kBack], uint32_t done) {
      int b = p.batch;
      uint32_t low = 0;
#pragma unroll
      for (int i = 0; i < kBack; ++i) {
        const uint32_t k = done + kBack * tid + i, e = entries - 1 - k;
        v[i] = -1;
        if (k >= entries) continue;
        if (i == 0 || e < low) {
          b = first_above(s.end, b, e);
          low = b ? s.end[b - 1] : 0u;
        }
        v[i] = p.table[b * p.table_stride + s.past[b] + (e - low)];
      }
    };
    load_entries(page, 0);
#pragma unroll 1
    for (uint32_t done = 0; done < entries; done += kBack * THREADS) {
      if (done + kBack * THREADS < entries) load_entries(next, done + kBack * THREADS);
      uint32_t at = top, all_of_wave = 0, pushed = 0;
#pragma unroll
      for (int i = 0; i < kBack; ++i) {
        const uint64_t those = __ballot(page[i] >= 0 && page[i] < p.pages);
        at += (uint32_t)__popcll(those & ((1ull << lane) - 1));
        all_of_wave += (uint32_t)__popcll(those);
      }
      if (lane == 0) waves[0][wave] = all_of_wave;
      lds_barrier();
#pragma unroll
      for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) at += waves[0][w];
        pushed += waves[0][w];
      }
#pragma unroll
      for (int i = 0; i < kBack; ++i) {
        if (page[i] < 0 || page[i] >= p.pages) continue;
        if (at < (uint32_t)p.capacity) p.free_pages[at] = page[i];
        ++at;
      }
#pragma unroll
      for (int i = 0; i < kBack; ++i) page[i] = next[i];
      top = min(top + pushed, (uint32_t)p.capacity);
      lds_barrier();
    }
    __syncthreads();  // (the stores: rows read them below)
  }

  // rows that fit, pages needed
  uint32_t need[PER], row_end[PER], needs = 0;
  bool fits[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    row = min(row + min(count[i], most), most);
    row_end[i] = row;
    fits[i] = row <= (uint32_t)p.rows && past[i] + count[i] <= all;
    need[i] = fits[i] ? ((past[i] + count[i] + cells) >> p.page_shift) - ((past[i] + cells) >> p.page_shift) : 0u;
    needs += need[i];
  }
  uint32_t none = 0, upto = needs, all_needs;
  sums_before<THREADS>(none, upto, all_needs, most, waves);
  uint32_t last = 0;  // pages taken up to this thread's last sequence that takes some
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    const uint32_t first = upto;
    upto += need[i];
    const bool served = fits[i] && (need[i] == 0 || upto <= top);
    if (served && need[i]) last = upto;
    if (b < p.batch) {
      p.lengths_out[b] = (int32_t)(past[i] + (served ? count[i] : 0u));
      p.past[b] = (int32_t)past[i];
      p.starts[b + 1] = (int32_t)min(row_end[i], (uint32_t)p.rows);
      if (FILL) s.end[b] = row_end[i], s.taken[b] = served ? first : kNotServed, s.past[b] = past[i];
    }
  }
  // (one atomic per wave: one per sequence, to the same word, took several us
  // for 4096 sequences)
#pragma unroll
  for (int i = 32; i > 0; i >>= 1) last = max(last, (uint32_t)__shfl_xor((int)last, i));
  if (lane == 0 && last) atomicMax(&last_taken, last);
  __syncthreads();
  if (tid == 0) {
    p.starts[0] = 0;
    p.free_count_out[0] = (int32_t)(top - last_taken);
  }
  if (!FILL) return;
#pragma unroll 2
  for (int t = tid; t < p.rows; t += THREADS) {
    Row r;
    const int b = first_above(s.end, p.batch, (uint32_t)t);
    if (b < p.batch && s.taken[b] != kNotServed)
      r = row_of(p, b, (uint32_t)t - (b ? s.end[b - 1] : 0u), s.past[b], s.taken[b], top);
    p.positions[t] = r.position;
    p.slots[t] = slot_of(p, r);
  }
}

// PER neighbours of an array of n, from `at`.
template <int PER>
__device__ __forceinline__ void load_some(int32_t (&v)[PER], const int32_t* x, int at, int n) {
  typedef int32_t some_t __attribute__((ext_vector_type(PER), aligned(4)));
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = 0;
  if (at + PER <= n) {
    const some_t y = *reinterpret_cast<const some_t*>(x + at);
    __builtin_memcpy(v, &y, sizeof(v));
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at + i < n) v[i] = x[at + i];
  }
}

// The rows, after k_cache_plan: each workgroup forms the sums again from what
// that left (a sequence is served if its new length has its count, and the
// needs of the served ones before it are all that counts for its pages).
// Every sequence marks its first row among the workgroup's, and a running
// maximum over the rows tells each its sequence; a search per row instead
// (12 dependent reads of LDS) took 13.1 us for 1000000 rows of 4096 sequences,
// this 7.9; 70001 rows of 300: 6.7 and 4.5.
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) k_cache_fill(AssignParams p) {
  __shared__ uint32_t starts[THREADS * PER], taken[THREADS * PER], pasts[THREADS * PER];
  __shared__ __attribute__((aligned(8))) uint16_t owner[kEach * THREADS];  // 1 + sequence
  __shared__ uint32_t waves[2][THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b0 = tid * PER;
  const uint32_t cells = (1u << p.page_shift) - 1;
  const int first = blockIdx.x * (kEach * THREADS);
  *reinterpret_cast<uint64_t*>(owner + kEach * tid) = 0;
  const uint32_t left = (uint32_t)p.free_count_out[0];
  int32_t past[PER], count[PER], length[PER], end[PER];
  load_some(past, p.past, b0, p.batch);
  load_some(count, p.counts, b0, p.batch);
  load_some(length, p.lengths_out, b0, p.batch);
  load_some(end, p.starts + 1, b0, p.batch);
  int32_t begin = b0 < p.batch ? p.starts[b0] : 0;
  uint32_t need[PER], needs = 0;
  bool served[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t c = (uint32_t)max(count[i], 0), n = (uint32_t)past[i];
    served[i] = (uint32_t)length[i] == n + c;
    need[i] = served[i] ? ((n + c + cells) >> p.page_shift) - ((n + cells) >> p.page_shift) : 0u;
    needs += need[i];
  }
  uint32_t none = 0, before = needs, all_needs;
  sums_before<THREADS>(none, before, all_needs, 0u, waves);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (begin < end[i] && begin < first + kEach * THREADS && end[i] > first) {
      owner[max(begin, first) - first] = (uint16_t)(b0 + i + 1);
      starts[b0 + i] = (uint32_t)begin, pasts[b0 + i] = (uint32_t)past[i];
      taken[b0 + i] = served[i] ? before : kNotServed;
    }
    begin = end[i];
    before += need[i];
  }
  __syncthreads();
  uint32_t own[kEach], most = 0;
  uint64_t four = *reinterpret_cast<const uint64_t*>(owner + kEach * tid);
#pragma unroll
  for (int i = 0; i < kEach; ++i) own[i] = most = max(most, (uint32_t)(four >> (16 * i)) & 0xFFFFu);
#define BGG_SCAN_STEP(MOVE, ROWS) most = max(most, from_lane<MOVE, ROWS>(most))
  BGG_SCAN_STEP(0x111, 0xF);  // (as in sums_before)
  BGG_SCAN_STEP(0x112, 0xF);
  BGG_SCAN_STEP(0x114, 0xF);
  BGG_SCAN_STEP(0x118, 0xF);
  BGG_SCAN_STEP(0x142, 0xA);
  BGG_SCAN_STEP(0x143, 0xC);
#undef BGG_SCAN_STEP
  if (lane == 63) waves[0][wave] = most;
  uint32_t so_far = __shfl_up(most, 1);
  if (lane == 0) so_far = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w)
    if (w < wave) so_far = max(so_far, waves[0][w]);

  const int t0 = first + kEach * tid, upto = min(p.starts[p.batch], p.rows);
  Row r[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = (int)max(own[i], so_far) - 1, t = t0 + i;
    if (t < upto && b >= 0 && taken[b] != kNotServed)
      r[i] = row_of(p, b, (uint32_t)t - starts[b], pasts[b], taken[b], left + all_needs);
  }
  typedef int32_t positions_t __attribute__((ext_vector_type(kEach), aligned(4)));
  typedef int64_t slots_t __attribute__((ext_vector_type(kEach), aligned(8)));
  positions_t x;
  slots_t y;
#pragma unroll
  for (int i = 0; i < kEach; ++i) x[i] = r[i].position, y[i] = slot_of(p, r[i]);
  if (t0 + kEach <= p.rows) {
    *reinterpret_cast<positions_t*>(p.positions + t0) = x;
    *reinterpret_cast<slots_t*>(p.slots + t0) = y;
  } else {
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (t0 + i < p.rows) p.positions[t0 + i] = x[i], p.slots[t0 + i] = y[i];
  }
}

template <int THREADS, int PER>
void launch_assign(AssignParams& p, hipStream_t s) {
  // The planning workgroup writes up to four rows per thread itself, more are a
  // launch of their own (64 sequences: 1024 rows in one launch 4.7 us, in two
  // 1.9 + 3.1 and the gap between them; 4096 rows 11.6 and 2.0 + 3.8 us).
  if (p.rows <= 4 * THREADS) {
    hipLaunchKernelGGL((k_cache_plan<THREADS, PER, true>), dim3(1), dim3(THREADS), 0, s, p);
    return;
  }
  hipLaunchKernelGGL((k_cache_plan<THREADS, PER, false>), dim3(1), dim3(THREADS), 0, s, p);
  hipLaunchKernelGGL((k_cache_fill<THREADS, PER>), dim3((unsigned)ceil_div(p.rows, kEach * THREADS)), dim3(THREADS), 0, s, p);
}

}  // namespace

extern "C" bgg_status bgg_cache_assign(const bgg_cache_desc* c, const bgg_assign_args* a, void* stream) {
  const bgg_status st = check_assign(c, a);
  if (st) return st;
  AssignParams p{};
  p.lengths = a->lengths_dev;
  p.counts = a->counts_dev;
  p.shared = a->shared_pages_dev;
  p.table = a->page_table_dev;
  p.table_stride = a->table_stride;
  p.free_pages = a->free_pages_dev;
  p.free_count = a->free_count_dev;
  p.lengths_out = a->lengths_out_dev;
  p.free_count_out = a->free_count_out_dev;
  p.past = a->past_dev;
  p.starts = a->starts_dev;
  p.positions = a->positions_dev;
  p.slots = a->slots_dev;
  p.batch = (int)a->batch;
  p.rows = (int)a->rows;
  p.width = (int)a->table_width;
  p.capacity = (int)a->free_capacity;
  p.pages = (int)c->pages;
  p.page_shift = __builtin_ctzll((unsigned long long)c->page_size);
  // Threads and sequences per thread: fewer waves meet at the barriers sooner
  // (64 sequences of a token each: 256 threads 2.7 us, 1024 3.7), more search
  // for the pages given back at a time (256 sequences, many of which end: 9.8
  // and 7.1 us); of 1000 sequences, one per thread 12.8 us, four 14.1.
  if (a->batch <= 256)
    launch_assign<256, 1>(p, (hipStream_t)stream);
  else if (a->batch <= 1024)
    launch_assign<1024, 1>(p, (hipStream_t)stream);
  else
    launch_assign<1024, 4>(p, (hipStream_t)stream);
  return hip_check("bgg_cache_assign");
}
