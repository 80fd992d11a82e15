// Rotary positions of new tokens and the append of their keys and values to
// a paged cache: pairs (u, w) of a head's first values turn by the angle
// a = position * frequency, (u cos a - w sin a, u sin a + w cos a).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bgg_cache.h"
#include "bgg_lowp.h"

using namespace bgg;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int64_t kTargetGroups = 1024;  // workgroups that the rows of few tokens are spread over
constexpr int64_t kMinRows = 8;          // rows of a workgroup at least (one to 47 tokens: 2, 4, 8 and
                                         // 16 rows within 0.2 us, 16 e4m3 tokens 2.8, 2.8, 2.9, 3.3)

struct RotaryParams {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_stride, q_out_stride, k_stride, v_stride;
  const int32_t* positions;
  const int64_t* slots;
  const float* freqs;
  float magnitude;
  void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  int64_t all_slots;
  const uint8_t* axis_of_pair;  // nullptr: one position per token
  int64_t axis_stride;
  int last_axis;
  int q_heads, kv_heads, head_dim, pairs, interleaved, page_shift, rows_per_group;
};

// cos and sin of position * frequency: the product (31 and 24 bits) and its
// remainder of 2 pi in 64 bits, then fp32 functions of at most pi.
__device__ __forceinline__ void angle_of(int32_t position, float freq, float* c, float* s) {
  const double a = (double)position * (double)freq;
  const double n = rint(a * 0.15915494309189533577);
  const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586232, a));
  sincosf((float)r, s, c);
}

// This workgroup's token: its cos and sin (times the magnitude) in LDS.
__device__ __forceinline__ void angles_to_lds(const RotaryParams& p, int64_t t, float* cs, float* sn) {
  if ((int)threadIdx.x < p.pairs) {
    float c, s;
    int32_t position = p.positions[t];
    if (p.axis_of_pair) {  // (all axes' positions are loaded along with the pair's axis)
      const int axis = p.axis_of_pair[threadIdx.x];
#pragma unroll
      for (int i = 1; i < BGG_MAX_AXES; ++i) {
        const int32_t other = p.positions[min(i, p.last_axis) * p.axis_stride + t];
        position = axis >= i ? other : position;
      }
    }
    angle_of(position, p.freqs[threadIdx.x], &c, &s);
    cs[threadIdx.x] = c * p.magnitude;
    sn[threadIdx.x] = s * p.magnitude;
  }
  __syncthreads();
}

// Row h of token t: its query heads, key heads, value heads.
struct Row {
  const uint16_t* src;
  void* dst;
  bool query, turns;
  float scale;
};
template <class C>
__device__ __forceinline__ Row row_of(const RotaryParams& p, int64_t t, int64_t slot, int h) {
  Row r;
  const int D = p.head_dim;
  r.query = h < p.q_heads;
  r.turns = h < p.q_heads + p.kv_heads;
  r.scale = 1.0f;
  if (r.query) {
    r.src = p.q + t * p.q_stride + (int64_t)h * D;
    r.dst = p.q_out + t * p.q_out_stride + (int64_t)h * D;
    return r;
  }
  const int kh = h - p.q_heads - (r.turns ? 0 : p.kv_heads);
  r.src = (r.turns ? p.k + t * p.k_stride : p.v + t * p.v_stride) + (int64_t)kh * D;
  const int64_t page = slot >> p.page_shift, cell = slot & ((int64_t(1) << p.page_shift) - 1);
  r.dst = (typename C::bits_t*)(r.turns ? p.k_cache : p.v_cache) +
          (((page * p.kv_heads + kh) << p.page_shift) + cell) * D;
  if constexpr (sizeof(typename C::bits_t) == 1) r.scale = (r.turns ? p.k_scale : p.v_scale)[kh];
  return r;
}

// Values of the rotated part that a thread holds next to each other start at
// multiples of 8 (16 bytes): R / 2 a multiple of 8 (halves) or R of 8
// (interleaved).
__device__ __forceinline__ void load8(const uint16_t* p, uint4& v) { v = *reinterpret_cast<const uint4*>(p); }
template <class T>
__device__ __forceinline__ void values8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = T::value((uint16_t)w[i]), v[2 * i + 1] = T::value((uint16_t)(w[i] >> 16));
}
template <class X>
__device__ __forceinline__ void store8(void* row, int at, const float (&v)[8]) {
  uint32_t w[4];
  if constexpr (sizeof(typename X::bits_t) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)X::bits(v[2 * i]) | ((uint32_t)X::bits(v[2 * i + 1]) << 16);
    *reinterpret_cast<uint4*>((uint16_t*)row + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (uint32_t)X::bits(v[4 * i]) | ((uint32_t)X::bits(v[4 * i + 1]) << 8) |
             ((uint32_t)X::bits(v[4 * i + 2]) << 16) | ((uint32_t)X::bits(v[4 * i + 3]) << 24);
    *reinterpret_cast<uint2*>((uint8_t*)row + at) = make_uint2(w[0], w[1]);
  }
}

// Eight pairs (halves) or four (interleaved), or eight or sixteen values
// past the rotated part, per thread and row: 16-byte loads and stores.  A
// thread keeps its place in the head and so its cos and sin, and goes
// through the rows blockIdx.y, its threads' share at a time.  Bound by HBM
// for long prompts (each value read and written once: 4095 tokens of 48 + 16
// heads of 128 bf16, 134 MB, 21.5 us warm and 29 us from cold caches, where a
// large copy moves 4.9 TB/s); for a few tokens by the chain position -> angle
// -> rows (2.5 us, of which 1.7 launch), so the rows are spread over
// workgroups.
template <class T, class C, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rotary_append(RotaryParams p) {
  __shared__ __attribute__((aligned(16))) float cs[kMaxPairs], sn[kMaxPairs];
  const int64_t t = blockIdx.x;
  const int D = p.head_dim, P = p.pairs;
  const int turning = HALF ? P / 8 : P / 4;             // units of the rotated part
  const int units = turning + (D - 2 * P) / 8;          // of a head
  const int unit = threadIdx.x % units, per = kThreads / units, mine = threadIdx.x / units;
  const int64_t slot = p.k ? p.slots[t] : -1;
  const bool stored = slot >= 0 && slot < p.all_slots;
  const int heads = p.q_heads + (stored ? 2 * p.kv_heads : 0);
  const int h_end = min(heads, ((int)blockIdx.y + 1) * p.rows_per_group);
  const bool turn = unit < turning;
  const int a = !turn ? 2 * P + 8 * (unit - turning) : 8 * unit, b = HALF && turn ? a + P : a;
  int h = blockIdx.y * p.rows_per_group + mine;
  const bool any = mine < per && h < h_end;
  Row r;
  uint4 ua, ub;
  if (any) {  // the first row's loads go out before the angles
    r = row_of<C>(p, t, slot, h);
    load8(r.src + a, ua);
    if (HALF) load8(r.src + b, ub);
  }
  angles_to_lds(p, t, cs, sn);
  if (!any) return;
  constexpr int N = HALF ? 8 : 4;
  float c[N], s[N];
  if (turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = cs[N * unit + i], s[i] = sn[N * unit + i];
  }
  for (;;) {
    const int next = h + per;
    Row rn;
    uint4 na, nb;
    if (next < h_end) {
      rn = row_of<C>(p, t, slot, next);
      load8(rn.src + a, na);
      if (HALF) load8(rn.src + b, nb);
    }
    float x[8], y[8];
    values8<T>(ua, x);
    if (HALF) values8<T>(ub, y);
    if (turn && r.turns) {
      if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = x[i], w = y[i];
          x[i] = u * c[i] - w * s[i];
          y[i] = u * s[i] + w * c[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = x[2 * i], w = x[2 * i + 1];
          x[2 * i] = u * c[i] - w * s[i];
          x[2 * i + 1] = u * s[i] + w * c[i];
        }
      }
    }
    if (r.query) {
      store8<T>(r.dst, a, x);
      if (HALF && turn) store8<T>(r.dst, b, y);
    } else {
      if constexpr (sizeof(typename C::bits_t) == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] /= r.scale;
        if (HALF)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] /= r.scale;
      }
      store8<C>(r.dst, a, x);
      if (HALF && turn) store8<C>(r.dst, b, y);
    }
    if (next >= h_end) break;
    h = next;
    r = rn;
    ua = na;
    if (HALF) ub = nb;
  }
}

// Any even rotary_dim: one pair or value per thread and step, two bytes at a
// time (4095 tokens as above with all of the head rotated but two values: 32
// us, in 16-byte units 21.5).  For rotated parts whose halves, or whose end,
// lie inside a 16-byte unit: a thread's pairs are then spread over other
// threads' units.  Multiples of 16 (interleaved: of 8) never come here.
template <class T, class C>
__global__ void __launch_bounds__(kThreads) k_rotary_append_any(RotaryParams p) {
  __shared__ float cs[kMaxPairs], sn[kMaxPairs];
  const int64_t t = blockIdx.x;
  const int64_t slot = p.k ? p.slots[t] : -1;
  const bool stored = slot >= 0 && slot < p.all_slots;
  const int heads = p.q_heads + (stored ? 2 * p.kv_heads : 0);
  const int h0 = blockIdx.y * p.rows_per_group, h1 = min(heads, h0 + p.rows_per_group);
  angles_to_lds(p, t, cs, sn);
  const int D = p.head_dim, P = p.pairs;
  const int steps = D - P;  // pairs, then the values past the rotated part
  for (int i = threadIdx.x; i < (h1 - h0) * steps; i += kThreads) {
    const int h = h0 + i / steps, j = i % steps;
    const Row r = row_of<C>(p, t, slot, h);
    const bool pair = j < P;
    const int a = !pair ? j + P : p.interleaved ? 2 * j : j;
    const int b = !pair ? a : p.interleaved ? a + 1 : a + P;
    float u = T::value(r.src[a]), w = T::value(r.src[b]);
    if (pair && r.turns) {
      const float c = cs[j], s = sn[j];
      const float nu = u * c - w * s;
      w = u * s + w * c;
      u = nu;
    }
    if (r.query) {
      uint16_t* dst = (uint16_t*)r.dst;
      dst[a] = T::bits(u);
      dst[b] = T::bits(w);
      continue;
    }
    if constexpr (sizeof(typename C::bits_t) == 1) {
      u /= r.scale;
      w /= r.scale;
    }
    typename C::bits_t* dst = (typename C::bits_t*)r.dst;
    dst[a] = C::bits(u);
    dst[b] = C::bits(w);
  }
}

template <class T, class C>
void launch_rotary(const RotaryParams& p, dim3 grid, hipStream_t s) {
  const dim3 block(kThreads);
  if (p.pairs % (p.interleaved ? 4 : 8))
    hipLaunchKernelGGL((k_rotary_append_any<T, C>), grid, block, 0, s, p);
  else if (p.interleaved)
    hipLaunchKernelGGL((k_rotary_append<T, C, false>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((k_rotary_append<T, C, true>), grid, block, 0, s, p);
}

// The call, its arguments checked.
bgg_status append(const char* who, const bgg_cache_desc* c, const bgg_rotary_args* a, const bgg_rotary_axes_args* x,
                  void* stream) {
  if (a->tokens == 0) return BGG_OK;
  RotaryParams p{};
  if (x) {
    p.axis_of_pair = x->axis_of_pair_dev;
    p.axis_stride = x->stride;
    p.last_axis = (int)x->axes - 1;
  }
  p.q = (const uint16_t*)a->q_dev;
  p.k = (const uint16_t*)a->k_dev;
  p.v = (const uint16_t*)a->v_dev;
  p.q_out = (uint16_t*)a->q_out_dev;
  p.q_stride = a->q_stride;
  p.q_out_stride = a->q_out_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.positions = a->positions_dev;
  p.slots = a->slots_dev;
  p.freqs = a->freqs_dev;
  p.magnitude = a->magnitude;
  p.k_cache = a->k_cache_dev;
  p.v_cache = a->v_cache_dev;
  p.k_scale = a->k_scale_dev;
  p.v_scale = a->v_scale_dev;
  p.all_slots = c->pages * c->page_size;
  p.q_heads = (int)a->q_heads;
  p.kv_heads = (int)c->kv_heads;
  p.head_dim = (int)c->head_dim;
  p.pairs = (int)a->rotary_dim / 2;
  p.interleaved = a->layout == BGG_ROTARY_INTERLEAVED;
  p.page_shift = __builtin_ctzll((unsigned long long)c->page_size);
  // rows over workgroups until these fill the GPU a few times over
  const int64_t rows = a->q_heads + (a->k_dev ? 2 * c->kv_heads : 0);
  const int64_t groups = std::max<int64_t>(1, std::min<int64_t>(ceil_div(rows, kMinRows), ceil_div(kTargetGroups, a->tokens)));
  p.rows_per_group = (int)ceil_div(rows, groups);
  const dim3 grid((unsigned)a->tokens, (unsigned)ceil_div(rows, p.rows_per_group));
  hipStream_t s = (hipStream_t)stream;
  const bool e4m3 = a->k_dev && c->type == BGG_TYPE_E4M3;
  if (a->type == BGG_TYPE_F16) {
    if (e4m3)
      launch_rotary<F16, E4M3>(p, grid, s);
    else
      launch_rotary<F16, F16>(p, grid, s);
  } else {
    if (e4m3)
      launch_rotary<BF16, E4M3>(p, grid, s);
    else
      launch_rotary<BF16, BF16>(p, grid, s);
  }
  return hip_check(who);
}

}  // namespace

extern "C" {

bgg_status bgg_rotary_append(const bgg_cache_desc* c, const bgg_rotary_args* a, void* stream) {
  const bgg_status st = check_rotary(c, a);
  return st ? st : append("bgg_rotary_append", c, a, nullptr, stream);
}

bgg_status bgg_rotary_append_axes(const bgg_cache_desc* c, const bgg_rotary_args* a, const bgg_rotary_axes_args* x,
                                  void* stream) {
  const bgg_status st = check_rotary_axes(c, a, x);
  return st ? st : append("bgg_rotary_append_axes", c, a, x, stream);
}

}  // extern "C"
