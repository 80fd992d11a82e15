// 16- and 8-bit element types of activations and caches on the device.
#pragma once
#include "bgg_device.h"

namespace bgg {

// Tags of the element types; bits() stores one value, value() reads one.
struct F16 {
  using bits_t = uint16_t;
  static __device__ __forceinline__ float value(uint16_t b) { return h2f(b); }
  static __device__ __forceinline__ uint16_t bits(float v) { return f2h(v); }
};
struct BF16 {
  using bits_t = uint16_t;
  static __device__ __forceinline__ float value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t bits(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  }
};
struct E4M3 {
  using bits_t = uint8_t;
  static __device__ __forceinline__ float value(uint8_t b) {
    return __builtin_amdgcn_cvt_f32_fp8((int)b, 0);
  }
  // cut to the largest finite value; NaN stays NaN
  static __device__ __forceinline__ uint8_t bits(float v) {
    const float c = v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v;
    return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, c, 0, false);
  }
};

}  // namespace bgg
