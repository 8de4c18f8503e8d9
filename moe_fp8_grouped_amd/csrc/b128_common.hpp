// The block format of the b128 calls: 128 e4m3fn elements share one e8m0
// scale s, which stands for 2^(s - 127); 255 is NaN.
#pragma once

#include "common.hpp"

namespace moe {
namespace b128 {

constexpr int kBlock = 128;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }   // NaN is the largest

// Scale code of a block from the bits of its largest magnitude: the smallest
// power of two, at least 2^-127, with amax <= 448 times it.  448 = 1.75 * 2^8,
// so amax = 1.f * 2^e takes 2^(e - 8) up to f = 0.75 and 2^(e - 7) above.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23);
  const uint32_t s = static_cast<uint32_t>(max(e - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), 0));
  return e == 255 ? 255u : amax == 0u ? 127u : s;
}

// 1 / scale, a power of two in float32's normal range for every code that
// scale_code gives (0 to 247); 0 for NaN, whose codes are all 0.
__device__ __forceinline__ float inverse(uint32_t code) { return __uint_as_float(code == 255u ? 0u : (254u - code) << 23); }

// The scale as a float: 2^(code - 127); code 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t code) {
  return __uint_as_float(code == 0u ? 0x00400000u : code == 255u ? 0x7fc00000u : code << 23);
}

// Eight values to codes.  v * inv is exact where it matters (a product that
// leaves float32's range downwards is far below half the smallest code), so
// the conversion's rounding, to nearest even, is the only one.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, hi, true);
  return inv == 0.0f ? make_uint2(0u, 0u) : make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
}

// One group's place among the local groups, by whole blocks of 128 rows.
struct GroupBlock {
  int g, m;                                  // the local group, and its rows
  int64_t row0;                              // its first local row
  int64_t block0;                            // its first block among all groups'
};

// The group that holds block b (every lane of the wave gets the answer), or
// g = -1 past the last.  Sizes below zero count as 0, rows past max_rows not
// at all.  `err` (or NULL) receives what is wrong with the sizes.
__device__ __forceinline__ GroupBlock find_block(const int32_t* __restrict__ sizes, int El, int64_t max_rows, int64_t b, int32_t* err) {
  const int lane = threadIdx.x & 63;
  int64_t rows = 0, blocks = 0;
  for (int base = 0; base < El; base += 64) {
    const int raw = base + lane < El ? sizes[base + lane] : 0;
    const int64_t size = raw < 0 ? 0 : raw;
    int64_t end = size;                      // inclusive scan of the sizes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t t = __shfl_up(end, o, 64);
      if (lane >= o) end += t;
    }
    const int64_t r0 = min(rows + end - size, max_rows), r1 = min(rows + end, max_rows);
    if (err) {
      if (raw < 0) raise_error(err, MOE_DEVERR_GROUP_SIZE);
      if (rows + end > max_rows) raise_error(err, MOE_DEVERR_ROWS);
    }
    const int64_t nb = (r1 - r0 + kBlock - 1) / kBlock;
    int64_t bend = nb;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t t = __shfl_up(bend, o, 64);
      if (lane >= o) bend += t;
    }
    const uint64_t has = __ballot(blocks + bend > b);
    if (has) {
      const int l = __builtin_ctzll(has);
      GroupBlock f;
      f.g = base + l;
      f.m = static_cast<int>(__shfl(r1 - r0, l, 64));
      f.row0 = __shfl(r0, l, 64);
      f.block0 = __shfl(blocks + bend - nb, l, 64);
      return f;
    }
    rows += __shfl(end, 63, 64);
    blocks += __shfl(bend, 63, 64);
  }
  return GroupBlock{-1, 0, 0, blocks};
}

}  // namespace b128
}  // namespace moe
