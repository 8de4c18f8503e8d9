// The 4-bit block format of the mx4 calls: 32 e2m1 elements share one e8m0
// scale.  An element's code is sign, two exponent bits, one mantissa bit:
// magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale code s stands for 2^(s-127),
// 255 for NaN.  Two codes a byte, the even element in the low half.
#pragma once

#include "common.hpp"

namespace moe {
namespace mx4 {

constexpr int kBlock = 32;

// Scale code of a block from the bits of its largest magnitude (a bfloat16 or
// float32 pattern's upper 16 bits give the same exponent field): the power of
// two that brings it into [4, 8), at least 2^-127; 2^0 for a block of zeros;
// NaN for a block with an element that is not finite.
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const uint32_t e = __float_as_uint(amax) >> 23;
  if (e >= 255u) return 255u;
  if (amax == 0.0f) return 127u;
  return e > 2u ? e - 2u : 0u;
}

// The scale as a float: 2^(code - 127); code 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t code) {
  return __uint_as_float(code == 0u ? 0x00400000u : code == 255u ? 0x7fc00000u : code << 23);
}

// Its reciprocal 2^(127 - code), exact; a NaN block multiplies by 0, so its
// codes are 0 (NaN and infinities included: encode() takes NaN to 0).
__device__ __forceinline__ float scale_inverse(uint32_t code) {
  return code == 255u ? 0.0f : __uint_as_float((254u - code) << 23);
}

// Nearest e2m1 code, ties to the even code, saturating at 6; NaN gives 0.
__device__ __forceinline__ uint32_t encode(float v) {
  const float a = fabsf(v);
  uint32_t c = 0;
  c += a > 0.25f;
  c += a >= 0.75f;
  c += a > 1.25f;
  c += a >= 1.75f;
  c += a > 2.5f;
  c += a >= 3.5f;
  c += a > 5.0f;
  return c | (a == a ? (__float_as_uint(v) >> 28) & 8u : 0u);
}

__device__ __forceinline__ float decode(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, f = c & 1u;
  const float a = e == 0 ? 0.5f * static_cast<float>(f)
                         : __uint_as_float(((126u + e) << 23) | (f << 22));
  return (c & 8u) ? -a : a;
}

}  // namespace mx4
}  // namespace moe
