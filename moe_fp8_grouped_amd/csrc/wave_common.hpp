// Sums and maxima over a wave, or over rows of sixteen lanes, in the vector
// unit: rows of 16 by shifts, then rows into rows (through LDS, as a shuffle goes,
// a chain of them takes most of a small kernel's time).
#pragma once

#include "common.hpp"

namespace moe {

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(none), static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float none, float v) {
  return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(none), __float_as_uint(v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double none, double v) {
  const uint64_t n = __double_as_longlong(none), b = __double_as_longlong(v);
  const uint32_t lo = dpp<CTRL, ROWS>(static_cast<uint32_t>(n), static_cast<uint32_t>(b));
  const uint32_t hi = dpp<CTRL, ROWS>(static_cast<uint32_t>(n >> 32), static_cast<uint32_t>(b >> 32));
  return __longlong_as_double(static_cast<int64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ float from_lane(float v, int lane) { return __uint_as_float(from_lane(__float_as_uint(v), lane)); }
__device__ __forceinline__ double from_lane(double v, int lane) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = from_lane(static_cast<uint32_t>(b), lane), hi = from_lane(static_cast<uint32_t>(b >> 32), lane);
  return __longlong_as_double(static_cast<int64_t>(hi) << 32 | lo);
}

// Over the wave, the same value for every lane.
template <class T, class F>
__device__ __forceinline__ T over_wave(T v, T none, const F& f) {
  v = f(v, dpp<0x111, 0xf>(none, v));        // row_shr 1, 2, 4, 8
  v = f(v, dpp<0x112, 0xf>(none, v));
  v = f(v, dpp<0x114, 0xf>(none, v));
  v = f(v, dpp<0x118, 0xf>(none, v));
  v = f(v, dpp<0x142, 0xa>(none, v));        // row_bcast 15 into rows 1 and 3, 31 into rows 2 and 3
  v = f(v, dpp<0x143, 0xc>(none, v));
  return from_lane(v, 63);
}
template <class T>
__device__ __forceinline__ T sum_of(T v) {
  return over_wave(v, T(0), [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float max_of(float v) {
  return over_wave(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  return over_wave(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// Over sixteen lanes, the same bits for each of them.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0xB1, 0xf>(0.0f, v);              // lane ^ 1, ^ 2, then halves and rows mirrored
  v += dpp<0x4E, 0xf>(0.0f, v);
  v += dpp<0x141, 0xf>(0.0f, v);
  v += dpp<0x140, 0xf>(0.0f, v);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<0xB1, 0xf>(0.0f, v));
  v = fmaxf(v, dpp<0x4E, 0xf>(0.0f, v));
  v = fmaxf(v, dpp<0x141, 0xf>(0.0f, v));
  v = fmaxf(v, dpp<0x140, 0xf>(0.0f, v));
  return v;
}

}  // namespace moe
