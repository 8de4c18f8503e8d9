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
  int row0;                                  // its first local row
  int block0;                                // its first block among all groups'
};

// Inclusive sum over the wave of values from 0 to cap, itself at most cap (which makes it the same in any order): rows of
// 16 by shifts, then rows into rows, in the vector unit.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_from(int v, int cap) {
  return min(v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false), cap);
}
__device__ __forceinline__ int wave_scan(int v, int cap) {
  v = add_from<0x111, 0xf>(v, cap);          // row_shr 1, 2, 4, 8
  v = add_from<0x112, 0xf>(v, cap);
  v = add_from<0x114, 0xf>(v, cap);
  v = add_from<0x118, 0xf>(v, cap);
  v = add_from<0x142, 0xa>(v, cap);          // row_bcast 15 into rows 1 and 3, 31 into rows 2 and 3
  return add_from<0x143, 0xc>(v, cap);
}

// The group that holds block b (every lane of the wave gets the answer), or
// g = -1 past the last.  Sizes below zero count as 0, rows past max_rows (at
// most 2^23) not at all.  `err` (or NULL) receives what is wrong with the sizes.
__device__ __forceinline__ GroupBlock find_block(const int32_t* __restrict__ sizes, int El, int max_rows, int b, int32_t* err) {
  const int lane = threadIdx.x & 63, cap = max_rows + 1;
  int rows = 0, blocks = 0;
  for (int base = 0; base < El; base += 64) {
    const int raw = base + lane < El ? sizes[base + lane] : 0;
    const int size = min(max(raw, 0), cap), before = lane == 0 ? rows : 0;
    const int end = wave_scan(min(size + before, cap), cap);               // rows up to this group's last
    const int up = __builtin_amdgcn_update_dpp(rows, end, 0x138, 0xf, 0xf, false);        // wave_shr 1: up to its first
    const int r0 = min(up, max_rows), r1 = min(end, max_rows);
    if (err) {
      if (raw < 0) raise_error(err, MOE_DEVERR_GROUP_SIZE);
      if (end > max_rows) raise_error(err, MOE_DEVERR_ROWS);
    }
    const int nb = (r1 - r0 + kBlock - 1) / kBlock;
    const int bend = blocks + wave_scan(nb, cap);                          // (fewer blocks than rows)
    const uint64_t has = __ballot(bend > b);
    if (has) {
      const int l = __builtin_ctzll(has);
      GroupBlock f;
      f.g = base + l;
      f.m = __builtin_amdgcn_readlane(r1 - r0, l);
      f.row0 = __builtin_amdgcn_readlane(r0, l);
      f.block0 = __builtin_amdgcn_readlane(bend - nb, l);
      return f;
    }
    rows = __builtin_amdgcn_readlane(end, 63);
    blocks = __builtin_amdgcn_readlane(bend, 63);
  }
  return GroupBlock{-1, 0, 0, blocks};
}

}  // namespace b128
}  // namespace moe
