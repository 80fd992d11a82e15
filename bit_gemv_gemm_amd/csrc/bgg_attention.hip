// Attention of one new token per sequence over a paged cache:
// s_t = scale q.k_t, out = sum_t e^(s_t) v_t / sum_t e^(s_t).
#include <hip/hip_runtime.h>

#include "bgg_cache.h"
#include "bgg_lowp.h"

using namespace bgg;

namespace {

struct AttnParams {
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  float* lse;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lengths;
  int64_t window, max_tokens;
  float scale;
  int pages, q_heads, kv_heads, page_shift;
};

// One wave per (query head, sequence): the tokens one after the other, the
// head's values spread over the lanes, running maximum and sum.
template <class T, class C, int D>
__global__ void __launch_bounds__(64) k_paged_attention(AttnParams p) {
  constexpr int N = (D + 63) / 64;
  const int lane = threadIdx.x, h = blockIdx.x;
  const int64_t b = blockIdx.y;
  const int kh = h / (p.q_heads / p.kv_heads);
  const int64_t len = p.lengths[b];
  const int64_t n = len < 0 ? 0 : len < p.max_tokens ? len : p.max_tokens;
  const int64_t lo = p.window > 0 && n > p.window ? n - p.window : 0;
  const float ks = p.k_scale ? p.k_scale[kh] : 1.0f, vs = p.v_scale ? p.v_scale[kh] : 1.0f;
  float q[N], acc[N], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int d = lane + 64 * i;
    q[i] = d < D ? T::value(p.q[b * p.q_stride + (int64_t)h * D + d]) : 0.0f;
    acc[i] = 0.0f;
  }
  const int64_t mask = (int64_t(1) << p.page_shift) - 1;
  for (int64_t t = lo; t < n; ++t) {
    const int page = p.table[b * p.table_stride + (t >> p.page_shift)];
    if (page < 0 || page >= p.pages) continue;
    const int64_t at = ((((int64_t)page * p.kv_heads + kh) << p.page_shift) + (t & mask)) * D;
    const auto* k = (const typename C::bits_t*)p.k_cache + at;
    const auto* v = (const typename C::bits_t*)p.v_cache + at;
    float s = 0.0f, vv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int d = lane + 64 * i;
      if (d < D) s = fmaf(q[i], C::value(k[d]), s);
      vv[i] = d < D ? C::value(v[d]) : 0.0f;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    s *= p.scale * ks;
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), f = expf(m - mn), e = expf(s - mn);
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = acc[i] * f + e * vv[i];
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int d = lane + 64 * i;
    if (d < D) p.out[b * p.out_stride + (int64_t)h * D + d] = T::bits(l > 0.0f || l != l ? acc[i] * vs / l : 0.0f);
  }
  if (p.lse && lane == 0) p.lse[b * p.q_heads + h] = m + logf(l);
}

template <class T, class C>
void launch_dim(const AttnParams& p, int64_t batch, int64_t head_dim, hipStream_t s) {
  const dim3 grid((unsigned)p.q_heads, (unsigned)batch), block(64);
  switch (head_dim) {
    case 64: hipLaunchKernelGGL((k_paged_attention<T, C, 64>), grid, block, 0, s, p); break;
    case 96: hipLaunchKernelGGL((k_paged_attention<T, C, 96>), grid, block, 0, s, p); break;
    case 128: hipLaunchKernelGGL((k_paged_attention<T, C, 128>), grid, block, 0, s, p); break;
    case 192: hipLaunchKernelGGL((k_paged_attention<T, C, 192>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((k_paged_attention<T, C, 256>), grid, block, 0, s, p); break;
  }
}

uint64_t counter_bytes(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  return align256(4ull * (uint64_t)batch * c->kv_heads * ceil_div(q_heads / c->kv_heads, 16));
}

}  // namespace

extern "C" {

size_t bgg_attention_workspace_size(const bgg_cache_desc* c, int64_t q_heads, int64_t batch) {
  if (check_cache(c) != BGG_OK || q_heads < 1 || q_heads > kMaxQHeads || q_heads % c->kv_heads ||
      batch < 1 || batch > kMaxBatch)
    return 0;
  return (size_t)counter_bytes(c, q_heads, batch);
}

bgg_status bgg_paged_attention(const bgg_cache_desc* c, const bgg_attention_args* a, void* stream) {
  bgg_status st = check_attention(c, a);
  if (st) return st;
  if (a->batch == 0) return BGG_OK;
  const size_t need = bgg_attention_workspace_size(c, a->q_heads, a->batch);
  if (a->workspace_bytes < need)
    return fail(BGG_ERR_BUFFER, "bgg_paged_attention: workspace has %zu bytes, needs %zu",
                a->workspace_bytes, need);
  AttnParams p{};
  p.q = (const uint16_t*)a->q_dev;
  p.out = (uint16_t*)a->out_dev;
  p.q_stride = a->q_stride;
  p.out_stride = a->out_stride;
  p.lse = a->lse_dev;
  p.k_cache = a->k_cache_dev;
  p.v_cache = a->v_cache_dev;
  p.k_scale = a->k_scale_dev;
  p.v_scale = a->v_scale_dev;
  p.table = a->page_table_dev;
  p.table_stride = a->table_stride;
  p.lengths = a->lengths_dev;
  p.window = a->window;
  p.max_tokens = a->table_width * c->page_size;
  p.scale = a->scale;
  p.pages = (int)c->pages;
  p.q_heads = (int)a->q_heads;
  p.kv_heads = (int)c->kv_heads;
  p.page_shift = __builtin_ctzll((unsigned long long)c->page_size);
  hipStream_t s = (hipStream_t)stream;
  const bool e4m3 = c->type == BGG_TYPE_E4M3;
  if (a->type == BGG_TYPE_F16) {
    if (e4m3)
      launch_dim<F16, E4M3>(p, a->batch, c->head_dim, s);
    else
      launch_dim<F16, F16>(p, a->batch, c->head_dim, s);
  } else {
    if (e4m3)
      launch_dim<BF16, E4M3>(p, a->batch, c->head_dim, s);
    else
      launch_dim<BF16, BF16>(p, a->batch, c->head_dim, s);
  }
  return hip_check("bgg_paged_attention");
}

}  // extern "C"
