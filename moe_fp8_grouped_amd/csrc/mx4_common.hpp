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

__device__ __forceinline__ float decode(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, f = c & 1u;
  const float a = e == 0 ? 0.5f * static_cast<float>(f)
                         : __uint_as_float(((126u + e) << 23) | (f << 22));
  return (c & 8u) ? -a : a;
}

// Four loads of 64 bytes a row, turned into four matrix-core fragments.  The
// fragment layout wants lane n + 16 g to hold chunk g (16 bytes) of row n, so
// a fragment loaded as it is asks for 16 bytes of another row with every lane,
// and the address unit takes the lanes one by one: 16 B a clock and CU,
// measured on data in L2, against 54 where four neighbouring lanes read 64
// bytes in a row.  So load i has lane 16 h + 4 m + c read chunk c of row
// 4 m + i of fragment h, and two 4 x 4 exchanges set it right: register
// against the lane's lowest two bits (i against c), then register against its
// highest two (c against h).
__device__ __forceinline__ void quad_exchange(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, bool b0, bool b1) {
  constexpr int kXor1 = 0xB1, kXor2 = 0x4E;      // quad_perm: lane ^ 1, lane ^ 2
#define MOE_QUAD(v, p) static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), p, 0xf, 0xf, true))
  const uint32_t x0 = MOE_QUAD(r0, kXor1), x1 = MOE_QUAD(r1, kXor1), x2 = MOE_QUAD(r2, kXor1), x3 = MOE_QUAD(r3, kXor1);
  const uint32_t t0 = b0 ? x1 : r0, t1 = b0 ? r1 : x0, t2 = b0 ? x3 : r2, t3 = b0 ? r3 : x2;
  const uint32_t y0 = MOE_QUAD(t0, kXor2), y1 = MOE_QUAD(t1, kXor2), y2 = MOE_QUAD(t2, kXor2), y3 = MOE_QUAD(t3, kXor2);
#undef MOE_QUAD
  r0 = b1 ? y2 : t0;
  r1 = b1 ? y3 : t1;
  r2 = b1 ? t2 : y0;
  r3 = b1 ? t3 : y1;
  const auto a = __builtin_amdgcn_permlane32_swap(r0, r2, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(r1, r3, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  r0 = c[0];
  r1 = c[1];
  r2 = d[0];
  r3 = d[1];
}
__device__ __forceinline__ void quad_exchange(uint4 (&w)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  quad_exchange(w[0].x, w[1].x, w[2].x, w[3].x, b0, b1);
  __builtin_amdgcn_sched_barrier(0);             // one word at a time: few registers beside the set's own
  quad_exchange(w[0].y, w[1].y, w[2].y, w[3].y, b0, b1);
  __builtin_amdgcn_sched_barrier(0);
  quad_exchange(w[0].z, w[1].z, w[2].z, w[3].z, b0, b1);
  __builtin_amdgcn_sched_barrier(0);
  quad_exchange(w[0].w, w[1].w, w[2].w, w[3].w, b0, b1);
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace mx4
}  // namespace moe
