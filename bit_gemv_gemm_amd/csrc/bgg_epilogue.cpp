// The epilogue's argument check, shared by the decode and prompt products.
#include "bgg_epilogue.h"

namespace bgg {

bgg_status epilogue_out(const char* who, const bgg_epilogue* ep, void* y, int64_t N, EpilogueOut* out) {
  if (!ep) return fail(BGG_ERR_NULL, "%s: NULL epilogue", who);
  if (ep->activation < BGG_ACT_NONE || ep->activation > BGG_ACT_GELU_TANH)
    return fail(BGG_ERR_FORMAT, "%s: unknown activation %d", who, (int)ep->activation);
  if (ep->reserved != 0) return fail(BGG_ERR_SHAPE, "%s: reserved must be 0", who);
  if (((uintptr_t)ep->bias_dev | (uintptr_t)ep->mul_dev | (uintptr_t)ep->residual_dev) & 1)
    return fail(BGG_ERR_BUFFER, "%s: misaligned epilogue operand", who);
  const int64_t most = int64_t(1) << 40;
  if (ep->mul_dev ? ep->mul_stride < N || ep->mul_stride > most : ep->mul_stride != 0)
    return fail(BGG_ERR_SHAPE, "%s: mul_stride %lld", who, (long long)ep->mul_stride);
  if (ep->residual_dev ? ep->residual_stride < N || ep->residual_stride > most : ep->residual_stride != 0)
    return fail(BGG_ERR_SHAPE, "%s: residual_stride %lld", who, (long long)ep->residual_stride);
  if ((ep->mul_dev && ep->mul_dev == y && ep->mul_stride != N) ||
      (ep->residual_dev && ep->residual_dev == y && ep->residual_stride != N))
    return fail(BGG_ERR_SHAPE, "%s: y as an operand has rows of N values", who);
  out->y = (uint16_t*)y;
  out->N = N;
  out->bias = (const uint16_t*)ep->bias_dev;
  out->mul = (const uint16_t*)ep->mul_dev;
  out->residual = (const uint16_t*)ep->residual_dev;
  out->mul_stride = ep->mul_stride;
  out->residual_stride = ep->residual_stride;
  out->act = ep->activation;
  // (a missing operand has address and stride 0)
  out->wide = N % 8 == 0 && ep->mul_stride % 8 == 0 && ep->residual_stride % 8 == 0 &&
              (((uintptr_t)y | (uintptr_t)ep->bias_dev | (uintptr_t)ep->mul_dev | (uintptr_t)ep->residual_dev) & 15) == 0;
  return BGG_OK;
}

}  // namespace bgg
