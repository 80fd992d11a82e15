// Rotary positions of new tokens and the append of their keys and values to
// a paged cache: pairs (u, w) of a head's first values turn by the angle
// a = position * frequency, (u cos a - w sin a, u sin a + w cos a).
#include <hip/hip_runtime.h>

#include "bgg_cache.h"
#include "bgg_lowp.h"

using namespace bgg;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

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
  int q_heads, kv_heads, head_dim, pairs, interleaved, page_shift;
};

// cos and sin of position * frequency: the product (31 and 24 bits) and its
// remainder of 2 pi in 64 bits, then fp32 functions of at most pi.
__device__ __forceinline__ void angle_of(int32_t position, float freq, float* c, float* s) {
  const double a = (double)position * (double)freq;
  const double n = rint(a * 0.15915494309189533577);
  const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586232, a));
  *c = cosf((float)r);
  *s = sinf((float)r);
}

// One workgroup per token: the token's cos and sin in LDS, then its heads'
// pairs and values one per thread and step.
template <class T, class C>
__global__ void __launch_bounds__(kThreads) k_rotary_append(RotaryParams p) {
  __shared__ float cs[kMaxPairs], sn[kMaxPairs];
  const int64_t t = blockIdx.x;
  if ((int)threadIdx.x < p.pairs) {
    float c, s;
    angle_of(p.positions[t], p.freqs[threadIdx.x], &c, &s);
    cs[threadIdx.x] = c * p.magnitude;
    sn[threadIdx.x] = s * p.magnitude;
  }
  __syncthreads();
  const int D = p.head_dim, P = p.pairs;
  const int steps = D - P;  // pairs, then the values past the rotated part
  const int64_t slot = p.k ? p.slots[t] : -1;
  const bool stored = slot >= 0 && slot < p.all_slots;
  const int heads = p.q_heads + (stored ? 2 * p.kv_heads : 0);
  for (int i = threadIdx.x; i < heads * steps; i += kThreads) {
    const int h = i / steps, j = i % steps;
    const bool is_q = h < p.q_heads, is_k = !is_q && h < p.q_heads + p.kv_heads;
    const int kh = is_q ? 0 : is_k ? h - p.q_heads : h - p.q_heads - p.kv_heads;
    const uint16_t* src = is_q ? p.q + t * p.q_stride + (int64_t)h * D
                          : is_k ? p.k + t * p.k_stride + (int64_t)kh * D
                                 : p.v + t * p.v_stride + (int64_t)kh * D;
    const bool pair = j < P;
    const int a = !pair ? j + P : p.interleaved ? 2 * j : j;
    const int b = !pair ? a : p.interleaved ? a + 1 : a + P;
    float u = T::value(src[a]), w = T::value(src[b]);
    if (pair && (is_q || is_k)) {
      const float c = cs[j], s = sn[j];
      const float nu = u * c - w * s;
      w = u * s + w * c;
      u = nu;
    }
    if (is_q) {
      uint16_t* dst = p.q_out + t * p.q_out_stride + (int64_t)h * D;
      dst[a] = T::bits(u);
      dst[b] = T::bits(w);
      continue;
    }
    if constexpr (sizeof(typename C::bits_t) == 1) {
      const float sc = (is_k ? p.k_scale : p.v_scale)[kh];
      u /= sc;
      w /= sc;
    }
    const int64_t page = slot >> p.page_shift, cell = slot & ((int64_t(1) << p.page_shift) - 1);
    typename C::bits_t* dst = (typename C::bits_t*)(is_k ? p.k_cache : p.v_cache) +
                              (((page * p.kv_heads + kh) << p.page_shift) + cell) * D;
    dst[a] = C::bits(u);
    dst[b] = C::bits(w);
  }
}

}  // namespace

extern "C" bgg_status bgg_rotary_append(const bgg_cache_desc* c, const bgg_rotary_args* a,
                                        void* stream) {
  bgg_status st = check_rotary(c, a);
  if (st) return st;
  if (a->tokens == 0) return BGG_OK;
  RotaryParams p{};
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
  const dim3 grid((unsigned)a->tokens), block(kThreads);
  hipStream_t s = (hipStream_t)stream;
  const bool e4m3 = a->k_dev && c->type == BGG_TYPE_E4M3;
  if (a->type == BGG_TYPE_F16) {
    if (e4m3)
      hipLaunchKernelGGL((k_rotary_append<F16, E4M3>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((k_rotary_append<F16, F16>), grid, block, 0, s, p);
  } else {
    if (e4m3)
      hipLaunchKernelGGL((k_rotary_append<BF16, E4M3>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((k_rotary_append<BF16, BF16>), grid, block, 0, s, p);
  }
  return hip_check("bgg_rotary_append");
}
