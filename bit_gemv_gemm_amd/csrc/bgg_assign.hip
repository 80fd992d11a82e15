// Page tables and slots of a serving batch's step, from the lengths of its
// sequences and a stack of free pages: prefix sums over the sequences, then
// a position and a slot per row.
//
// Two parts.  plan() is one workgroup's: pages given back, who is served,
// the new lengths (sums over up to 4096 sequences, in 32 bits: the call
// bounds what they add up to).  fill() writes the rows; each row looks its
// sequence up in the sums (in LDS, by halving) and takes its page from the
// table or, where the page is new, straight from the stack, so no row waits
// for another's entry of the table.  Both are bound by the chain of dependent
// loads (lengths -> sums -> table -> slot) for a decode step, and fill() by
// the 12 bytes written per row for long prompts.
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
  int batch, rows, width, capacity, pages, page_shift, rows_per_group;
};

constexpr uint32_t kNotServed = 0xFFFFFFFFu;
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

// Rows first .. end - 1, EACH neighbours per thread: one looks its sequence
// up, the others look on from there, and their page numbers are loaded
// together.  `top` is the height of the stack before pages were taken.
template <int THREADS, int EACH, int N>
__device__ __forceinline__ void fill(const AssignParams& p, const Sums<N>& s, int first, int end, uint32_t top) {
  typedef int32_t positions_t __attribute__((ext_vector_type(EACH), aligned(4)));
  typedef int64_t slots_t __attribute__((ext_vector_type(EACH), aligned(8)));
  const int cells = (1 << p.page_shift) - 1;
#pragma unroll 1
  for (int t = first + EACH * (int)threadIdx.x; t < end; t += EACH * THREADS) {
    int32_t position[EACH], page[EACH];
    int32_t* cell[EACH];
    bool fresh[EACH];
    int b = -1;
    uint32_t before = 0, upto = 0, taken = kNotServed, past = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (i == 0 || (b < p.batch && upto <= (uint32_t)(t + i))) {
        b += 1 + first_above(s.end + (b + 1), p.batch - (b + 1), (uint32_t)(t + i));
        if (b < p.batch) before = b ? s.end[b - 1] : 0u, upto = s.end[b], taken = s.taken[b], past = s.past[b];
      }
      position[i] = 0, page[i] = -1, fresh[i] = false;
      cell[i] = nullptr;
      if (b < p.batch && taken != kNotServed && t + i < end) {
        position[i] = (int32_t)(past + (uint32_t)(t + i) - before);
        const int entry = position[i] >> p.page_shift, held = (int)((past + cells) >> p.page_shift);
        cell[i] = p.table + b * p.table_stride + entry;
        fresh[i] = entry >= held;
        page[i] = *(fresh[i] ? p.free_pages + (top - 1 - (taken + (uint32_t)(entry - held))) : cell[i]);
      }
    }
    int64_t slot[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      // (a new page's first token is always new)
      if (fresh[i] && (position[i] & cells) == 0) *cell[i] = page[i];
      slot[i] = page[i] >= 0 && page[i] < p.pages ? ((int64_t)page[i] << p.page_shift) + (position[i] & cells) : -1;
    }
    if (t + EACH <= end) {
      positions_t x;
      slots_t y;
#pragma unroll
      for (int i = 0; i < EACH; ++i) x[i] = position[i], y[i] = slot[i];
      *reinterpret_cast<positions_t*>(p.positions + t) = x;
      *reinterpret_cast<slots_t*>(p.slots + t) = y;
    } else {
#pragma unroll
      for (int i = 0; i < EACH; ++i)
        if (t + i < end) p.positions[t + i] = position[i], p.slots[t + i] = slot[i];
    }
  }
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
#pragma unroll 1
    for (uint32_t done = 0; done < entries; done += kBack * THREADS) {
      // (kBack neighbours per thread, loaded together)
      int32_t page[kBack];
      int b = p.batch;
      uint32_t low = 0;
#pragma unroll
      for (int i = 0; i < kBack; ++i) {
        const uint32_t k = done + kBack * tid + i, e = entries - 1 - k;
        page[i] = -1;
        if (k >= entries) continue;
        if (i == 0 || e < low) {
          b = first_above(s.end, b, e);
          low = b ? s.end[b - 1] : 0u;
        }
        page[i] = p.table[b * p.table_stride + s.past[b] + (e - low)];
      }
      uint32_t at = top, all_of_wave = 0, pushed = 0;
#pragma unroll
      for (int i = 0; i < kBack; ++i) {
        const uint64_t those = __ballot(page[i] >= 0 && page[i] < p.pages);
        at += (uint32_t)__popcll(those & ((1ull << lane) - 1));
        all_of_wave += (uint32_t)__popcll(those);
      }
      if (lane == 0) waves[0][wave] = all_of_wave;
      __syncthreads();
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
      top = min(top + pushed, (uint32_t)p.capacity);
      __syncthreads();  // (also the stores: rows read them below)
    }
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
  // (one atomic per wave: of 64 lanes each it took SPLIT)
#pragma unroll
  for (int i = 32; i > 0; i >>= 1) last = max(last, (uint32_t)__shfl_xor((int)last, i));
  if (lane == 0 && last) atomicMax(&last_taken, last);
  __syncthreads();
  if (tid == 0) {
    p.starts[0] = 0;
    p.free_count_out[0] = (int32_t)(top - last_taken);
  }
  if (FILL) fill<THREADS, 1>(p, s, 0, p.rows, top);
}

// The rows, after k_cache_plan: each workgroup forms the sums again from what
// that left (a sequence is served if its new length has its count, and the
// needs of the served ones before it are all that counts for its pages).
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) k_cache_fill(AssignParams p) {
  __shared__ Sums<THREADS * PER> s;
  __shared__ uint32_t waves[2][THREADS / 64];
  const int tid = threadIdx.x;
  const uint32_t cells = (1u << p.page_shift) - 1;
  uint32_t need[PER], needs = 0;
  bool served[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    need[i] = 0;
    served[i] = false;
    if (b < p.batch) {
      const uint32_t past = (uint32_t)p.past[b], c = (uint32_t)max(p.counts[b], 0);
      served[i] = (uint32_t)p.lengths_out[b] == past + c;
      if (served[i]) need[i] = ((past + c + cells) >> p.page_shift) - ((past + cells) >> p.page_shift);
      s.end[b] = (uint32_t)p.starts[b + 1];
      s.past[b] = past;
    }
    needs += need[i];
  }
  uint32_t none = 0, first = needs, all_needs;
  sums_before<THREADS>(none, first, all_needs, 0u, waves);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b < p.batch) s.taken[b] = served[i] ? first : kNotServed;
    first += need[i];
  }
  __syncthreads();
  const int t0 = blockIdx.x * p.rows_per_group;
  fill<THREADS, 4>(p, s, t0, min(p.rows, t0 + p.rows_per_group), (uint32_t)p.free_count_out[0] + all_needs);
}

// Rows that the planning workgroup writes itself; more are a launch of their
// own, of kGroupRows rows per workgroup.
constexpr int kOwnRows = 4096, kGroupRows = 4096;

template <int THREADS, int PER>
void launch_assign(AssignParams& p, hipStream_t s) {
  if (p.rows <= kOwnRows) {
    hipLaunchKernelGGL((k_cache_plan<THREADS, PER, true>), dim3(1), dim3(THREADS), 0, s, p);
    return;
  }
  hipLaunchKernelGGL((k_cache_plan<THREADS, PER, false>), dim3(1), dim3(THREADS), 0, s, p);
  p.rows_per_group = kGroupRows;
  hipLaunchKernelGGL((k_cache_fill<THREADS, PER>), dim3((unsigned)ceil_div(p.rows, kGroupRows)), dim3(THREADS), 0, s, p);
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
  if (a->batch <= 256)
    launch_assign<256, 1>(p, (hipStream_t)stream);
  else
    launch_assign<1024, 4>(p, (hipStream_t)stream);
  return hip_check("bgg_cache_assign");
}
