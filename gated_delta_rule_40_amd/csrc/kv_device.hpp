// kv_device.hpp -- device helpers of the 8-bit key/value cache: e4m3 codes
// (OCP) and their power-of-two scales.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

constexpr float kE4m3Max = 448.0f;  // 1.75 * 2^8
constexpr int kMinScaleExp = -100;

// Smallest power of two s >= 2^-100 with amax <= 448 s, from the bits of amax
// (finite, >= 0): 448 = 1.75 * 2^8, so the exponent drops by 8, or by 7 where
// the significand of amax is above 1.75.  Subnormal amax falls to the floor.
__device__ __forceinline__ float e4m3_scale(float amax) {
  const unsigned u = __builtin_bit_cast(unsigned, amax);
  const int k = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __builtin_bit_cast(float, static_cast<unsigned>(max(k, kMinScaleExp) + 127) << 23);
}

// 1 / s for a power of two s in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float s) {
  return __builtin_bit_cast(float, 0x7f000000u - __builtin_bit_cast(unsigned, s));
}

// |x| if finite, else 0: what counts for a page's scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = __builtin_fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;  // false for NaN too
}

// e4m3 codes of two scaled values: round to nearest even, infinities to
// +-448 (fmin/fmax would turn NaN into a bound, comparisons keep it).
__device__ __forceinline__ unsigned e4m3_pair(float x, float y) {
  x = x > kE4m3Max ? kE4m3Max : x < -kE4m3Max ? -kE4m3Max : x;
  y = y > kE4m3Max ? kE4m3Max : y < -kE4m3Max ? -kE4m3Max : y;
  return static_cast<unsigned>(__builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false)) & 0xffffu;
}

__device__ __forceinline__ float e4m3_value(uint8_t code) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(code), 0);
}

}  // namespace gdr
