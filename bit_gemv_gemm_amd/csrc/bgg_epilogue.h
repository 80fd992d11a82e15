// Where the products put their results: y as it is, or through an epilogue,
// y = act(sum + bias) * mul + residual in fp32 with one rounding to fp16.
// The kernels are those of the plain products, with the output as a template
// argument; the epilogue costs its operands' bytes and little else (down
// 5120x17408 at one token onto a residual 6.77 us against 6.66, gate
// 17408x5120 at 16 tokens with SILU and a multiplier 22.5 against 21.5, at
// 4096 tokens 633 against 611, of which reading the multiplier is 23).
#pragma once
#include <cmath>

#include "bgg_device.h"

namespace bgg {

// y[m][n] = fp16(sum)
struct PlainOut {
  uint16_t* __restrict__ y;
  int64_t N;
  struct Operands {};
  __device__ __forceinline__ Operands load(int64_t, int64_t) const { return Operands{}; }
  __device__ __forceinline__ void store(int64_t m, int64_t n, float v, const Operands&) const {
    y[m * N + n] = f2h(v);
  }
};

// act(v).  1 / (1 + e) by the reciprocal instruction (one unit of fp32);
// 1 + erf(u) = erfc(-u) and (1 + tanh(u)) / 2 = 1 / (1 + e^(-2 u)), which do
// not cancel on the negative side.
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if (ACT == BGG_ACT_RELU) return v < 0.0f ? 0.0f : v;  // (a NaN stays)
  if (ACT == BGG_ACT_RELU2) return v < 0.0f ? 0.0f : v * v;
  if (ACT == BGG_ACT_SILU) return v * __builtin_amdgcn_rcpf(1.0f + __expf(-v));
  if (ACT == BGG_ACT_GELU) return 0.5f * v * erfcf(v * -0.7071067811865475f);
  if (ACT == BGG_ACT_GELU_TANH)
    return v * __builtin_amdgcn_rcpf(1.0f + __expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
  return v;
}

// The epilogue's operands of one value are loaded where its sum is about to
// arrive (load), so that their latency passes beside the last atomics or
// matrix operations, and applied when it has (store).  y may be mul or
// residual itself: each value is read before it is written, by the thread
// that writes it (where K is split over workgroups, by every workgroup
// before its arrival, and the last one writes).
struct EpilogueOut {
  uint16_t* y;
  int64_t N;
  const uint16_t *bias, *mul, *residual;
  int64_t mul_stride, residual_stride;
  int act;
  int wide;  // every row of y and of the operands starts on 16 bytes, N % 8 == 0
  struct Operands {
    uint16_t bias, mul, residual;
  };
  __device__ __forceinline__ Operands load(int64_t m, int64_t n) const {
    Operands o{0, 0x3C00, 0};
    if (bias) o.bias = bias[n];
    if (mul) o.mul = mul[m * mul_stride + n];
    if (residual) o.residual = residual[m * residual_stride + n];
    return o;
  }
  template <int ACT>
  __device__ __forceinline__ float value_of(float v, const Operands& o) const {
    if (bias) v += h2f(o.bias);
    v = activate<ACT>(v);
    if (mul) v *= h2f(o.mul);
    if (residual) v += h2f(o.residual);
    return v;
  }
  __device__ __forceinline__ float value(float v, const Operands& o) const {
    switch (act) {
      case BGG_ACT_RELU: return value_of<BGG_ACT_RELU>(v, o);
      case BGG_ACT_RELU2: return value_of<BGG_ACT_RELU2>(v, o);
      case BGG_ACT_SILU: return value_of<BGG_ACT_SILU>(v, o);
      case BGG_ACT_GELU: return value_of<BGG_ACT_GELU>(v, o);
      case BGG_ACT_GELU_TANH: return value_of<BGG_ACT_GELU_TANH>(v, o);
      default: return value_of<BGG_ACT_NONE>(v, o);
    }
  }
  __device__ __forceinline__ void store(int64_t m, int64_t n, float v, const Operands& o) const {
    y[m * N + n] = f2h(value(v, o));
  }
};

// BGG_OK and *out (device view, y included) for a checked call's epilogue.
bgg_status epilogue_out(const char* who, const bgg_epilogue* ep, void* y, int64_t N, EpilogueOut* out);

}  // namespace bgg
