// moe_quantize_rows_mx4, moe_quantize_weights_mx4, moe_dequantize_rows_mx4:
// to and from the microscaled 4-bit format (mx4_common.hpp).  The scale is a
// power of two and the values are bfloat16, so v / scale is exact and the
// only rounding is the one to e2m1.
#include "mx4_common.hpp"
#include "quant_common.hpp"

namespace moe {
namespace {
using namespace mx4;

// Four lanes hold one block, eight elements each.
template <bool SILU>
__global__ __launch_bounds__(256) void quantize_rows_mx4_kernel(const uint16_t* __restrict__ x,
                                                                const uint16_t* __restrict__ x_up, int64_t ldx,
                                                                int64_t R, int64_t C, uint8_t* __restrict__ q,
                                                                int64_t ldq, uint8_t* __restrict__ scale, int64_t lds) {
  const int64_t cpr = C >> 3;                // chunks of eight a row: a multiple of 4
  const int64_t total = R * cpr;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / cpr, c = i - r * cpr;
    float v[8];
    const Bf16x8 a{*reinterpret_cast<const uint4*>(x + r * ldx + 8 * c)};
    if (SILU) {
      const Bf16x8 b{*reinterpret_cast<const uint4*>(x_up + r * ldx + 8 * c)};
      float av[8], bv[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) { av[u] = a.get(u); bv[u] = b.get(u); }
      silu_mul8(av, bv, v);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = a.get(u);
    }
    uint32_t top = 0;                        // magnitudes' bits: NaN and infinity are the largest
#pragma unroll
    for (int u = 0; u < 8; ++u) top = max(top, __float_as_uint(v[u]) & 0x7fffffffu);
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1, MOE_WAVE)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2, MOE_WAVE)));
    const uint32_t s = scale_code(__uint_as_float(top));
    const float inv = scale_inverse(s);
    uint32_t w = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) w |= encode(v[u] * inv) << (4 * u);
    *reinterpret_cast<uint32_t*>(q + r * ldq + 4 * c) = w;
    if ((c & 3) == 0) scale[r * lds + (c >> 2)] = static_cast<uint8_t>(s);
  }
}

// A thread takes one block of 32 along K of one output channel.
__global__ __launch_bounds__(256) void quantize_weights_mx4_kernel(const uint16_t* __restrict__ w, int64_t K, int64_t N,
                                                                   uint8_t* __restrict__ q,
                                                                   uint8_t* __restrict__ scale, int64_t total) {
  const int64_t kb = K / kBlock;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t n = i % N, eb = i / N;     // neighbouring threads: neighbouring columns
    const int64_t b = eb % kb, e = eb / kb;
    const uint16_t* p = w + (e * K + b * kBlock) * N + n;
    float v[kBlock];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kBlock; ++u) {
      v[u] = bf16_to_f32(p[u * N]);
      top = max(top, __float_as_uint(v[u]) & 0x7fffffffu);
    }
    const uint32_t s = scale_code(__uint_as_float(top));
    const float inv = scale_inverse(s);
    uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < kBlock; ++u) o[u >> 3] |= encode(v[u] * inv) << (4 * (u & 7));
    const int64_t row = e * N + n;
    *reinterpret_cast<uint4*>(q + row * (K / 2) + 16 * b) = make_uint4(o[0], o[1], o[2], o[3]);
    scale[row * kb + b] = static_cast<uint8_t>(s);
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void dequantize_rows_mx4_kernel(const uint8_t* __restrict__ q, int64_t ldq,
                                                                  const uint8_t* __restrict__ scale, int64_t lds,
                                                                  int64_t R, int64_t C, void* __restrict__ out,
                                                                  int64_t ldo) {
  const int64_t cpr = C >> 3;
  const int64_t total = R * cpr;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / cpr, c = i - r * cpr;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(q + r * ldq + 4 * c);
    const float s = scale_value(scale[r * lds + (c >> 2)]);
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = decode((w >> (4 * u)) & 15u) * s;
    if (BF16) {
      uint32_t o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)            // two bits of mantissa: the rounding is exact
        o[u] = f32_to_bf16(v[2 * u]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * u + 1])) << 16);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + r * ldo + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + r * ldo + 8 * c);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

unsigned grid_for(int64_t items) {
  const int64_t b = moe_cdiv(items, 256);
  return static_cast<unsigned>(b < 1 ? 1 : b > 16384 ? 16384 : b);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace moe

extern "C" int moe_quantize_rows_mx4(const void* x, const void* x_up, int64_t ldx, int act, int64_t R, int64_t C,
                                     uint8_t* q, int64_t ldq, uint8_t* scale, int64_t lds, void* stream) {
  if (R < 0 || C <= 0 || C % 32 || ldx < C || ldx % 8 || ldq < C / 2 || ldq % 16 || lds < C / 32) return MOE_ERR_SHAPE;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SILU_MUL) return MOE_ERR_UNSUPPORTED;
  if (act == MOE_ACT_NONE && x_up) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!x || !q || !scale || (act == MOE_ACT_SILU_MUL && !x_up)) return MOE_ERR_NULL;
  if (!moe::aligned(x, 16) || !moe::aligned(x_up, 16) || !moe::aligned(q, 16)) return MOE_ERR_SHAPE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const uint16_t *xa = static_cast<const uint16_t*>(x), *xb = static_cast<const uint16_t*>(x_up);
  const unsigned grid = moe::grid_for(R * (C / 8));
  if (act == MOE_ACT_SILU_MUL)
    moe::quantize_rows_mx4_kernel<true><<<grid, 256, 0, st>>>(xa, xb, ldx, R, C, q, ldq, scale, lds);
  else
    moe::quantize_rows_mx4_kernel<false><<<grid, 256, 0, st>>>(xa, xb, ldx, R, C, q, ldq, scale, lds);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_quantize_weights_mx4(const void* w, int64_t E, int64_t K, int64_t N, uint8_t* q, uint8_t* scale,
                                        void* stream) {
  if (E < 0 || K <= 0 || K % 32 || N <= 0 || N % 16) return MOE_ERR_SHAPE;
  if (E == 0) return MOE_OK;
  if (!w || !q || !scale) return MOE_ERR_NULL;
  if (!moe::aligned(w, 16) || !moe::aligned(q, 16)) return MOE_ERR_SHAPE;
  const int64_t total = E * (K / 32) * N;
  moe::quantize_weights_mx4_kernel<<<moe::grid_for(total), 256, 0, static_cast<hipStream_t>(stream)>>>(
      static_cast<const uint16_t*>(w), K, N, q, scale, total);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_dequantize_rows_mx4(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds, int64_t R,
                                       int64_t C, int out_dtype, void* out, int64_t ldo, void* stream) {
  if (R < 0 || C <= 0 || C % 32 || ldq < C / 2 || ldq % 16 || lds < C / 32 || ldo < C || ldo % 8) return MOE_ERR_SHAPE;
  if (out_dtype == MOE_DTYPE_DEFAULT) out_dtype = MOE_BF16;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!q || !scale || !out) return MOE_ERR_NULL;
  if (!moe::aligned(q, 16) || !moe::aligned(out, 16)) return MOE_ERR_SHAPE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const unsigned grid = moe::grid_for(R * (C / 8));
  if (out_dtype == MOE_BF16)
    moe::dequantize_rows_mx4_kernel<true><<<grid, 256, 0, st>>>(q, ldq, scale, lds, R, C, out, ldo);
  else
    moe::dequantize_rows_mx4_kernel<false><<<grid, 256, 0, st>>>(q, ldq, scale, lds, R, C, out, ldo);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
