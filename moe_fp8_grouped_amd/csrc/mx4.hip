// moe_quantize_rows_mx4, moe_quantize_weights_mx4, moe_dequantize_rows_mx4:
// to and from the microscaled 4-bit format (mx4_common.hpp).  The scale is a
// power of two and the values are bfloat16, so v / scale is exact and the
// only rounding is the one to e2m1.
#include "mx4_common.hpp"
#include "quant_common.hpp"

namespace moe {
namespace {
using namespace mx4;

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Read once here, and not kept in the caches: 8 experts of 7168 by 2048 to
// codes and back 114 us instead of 131, 8192 rows of 7168 54 instead of 60.
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p)));
}

// Eight values to codes: v / 2^(s - 127), to the nearest even, saturating; a
// block that is not finite has codes 0.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t s) {
  const float sv = scale_value(s);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sv, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sv, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sv, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sv, 3);
  return s == 255u ? 0u : w;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }   // NaN is the largest

// Four lanes hold one block, eight elements each; a wave takes 64 such chunks
// of kRowsAWave rows, its loads first.  Memory bounds it: 8192 rows of 7168 to
// codes and back 52 us, 5.1 TB/s (a flat loop with a division a chunk and the
// codes from comparisons: 93).
constexpr int kRowsAWave = 4;

template <bool SILU>
__global__ __launch_bounds__(256) void quantize_rows_mx4_kernel(const uint16_t* __restrict__ x,
                                                                const uint16_t* __restrict__ x_up, int64_t ldx,
                                                                int64_t R, int64_t C, uint8_t* __restrict__ q,
                                                                int64_t ldq, uint8_t* __restrict__ scale, int64_t lds) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
  if (8 * c >= C) return;                    // (whole blocks: a row's chunks are a multiple of 4)
  const int64_t step = static_cast<int64_t>(gridDim.y) * 4;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * 4 + (threadIdx.x >> 6); r0 < R; r0 += step * kRowsAWave) {
    uint4 a[kRowsAWave], b[SILU ? kRowsAWave : 1];
#pragma unroll
    for (int u = 0; u < kRowsAWave; ++u) {
      const int64_t r = min(r0 + u * step, R - 1);
      a[u] = load_once(x + r * ldx + 8 * c);
      if constexpr (SILU) b[u] = load_once(x_up + r * ldx + 8 * c);
    }
#pragma unroll
    for (int u = 0; u < kRowsAWave; ++u) {
      const int64_t r = r0 + u * step;
      if (r >= R) break;
      float v[8];
      const Bf16x8 av{a[u]};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = av.get(i);
      if constexpr (SILU) {
        const Bf16x8 bv{b[u]};
        float g[8], h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) { g[i] = v[i]; h[i] = bv.get(i); }
        silu_mul8(g, h, v);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
      top = max(top, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(top), 0xB1, 0xf, 0xf, true)));   // lane ^ 1
      top = max(top, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(top), 0x4E, 0xf, 0xf, true)));   // lane ^ 2
      const uint32_t s = scale_code(__uint_as_float(top));
      *reinterpret_cast<uint32_t*>(q + r * ldq + 4 * c) = encode8(v, s);
      if ((c & 3) == 0) scale[r * lds + (c >> 2)] = static_cast<uint8_t>(s);
    }
  }
}

// A workgroup takes 128 output channels by 256 along K.  A lane reads 32
// elements of two neighbouring channels (a wave 256 bytes of a row of w), and
// the codes go through LDS, so that a channel's eight blocks leave as one
// 128-byte line.  Memory bounds it: 8 experts of 7168 by 2048 to codes and
// back 104 us, 5.1 TB/s (a thread a block, its 16 bytes written where they are
// formed, 64 channels apart: 177).
constexpr int kTileN = 128, kTileB = 8, kTilePitch = kTileB * 16 + 16;

__global__ __launch_bounds__(256) void quantize_weights_mx4_kernel(const uint16_t* __restrict__ w, int64_t E, int64_t K,
                                                                   int64_t N, uint8_t* __restrict__ q,
                                                                   uint8_t* __restrict__ scale) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[kTileN * kTilePitch];
  __shared__ __attribute__((aligned(16))) uint8_t sc[kTileN][kTileB];
  const int64_t kb = K / kBlock, n0 = static_cast<int64_t>(blockIdx.x) * kTileN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n = n0 + 2 * lane;           // (N is a multiple of 16: both channels exist, or neither)
  for (int64_t e = blockIdx.z; e < E; e += gridDim.z)
    for (int64_t b0 = static_cast<int64_t>(blockIdx.y) * kTileB; b0 < kb; b0 += static_cast<int64_t>(gridDim.y) * kTileB) {
      for (int j = wave; j < kTileB && b0 + j < kb; j += 4) {
        if (n >= N) continue;
        const uint16_t* p = w + (e * K + (b0 + j) * kBlock) * N + n;
        uint32_t pair[kBlock];
#pragma unroll
        for (int u = 0; u < kBlock; ++u) pair[u] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p + u * N));
        uint32_t top[2] = {0, 0}, o[2][4];
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {   // bfloat16 magnitudes order as their bits do
          top[0] = max(top[0], (pair[u] << 16) & 0x7fffffffu);
          top[1] = max(top[1], pair[u] & 0x7fff0000u);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t s = scale_code(__uint_as_float(top[h]));
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = __uint_as_float(h ? pair[8 * g + u] & 0xffff0000u : pair[8 * g + u] << 16);
            o[h][g] = encode8(v, s);
          }
          *reinterpret_cast<uint4*>(codes + (2 * lane + h) * kTilePitch + 16 * j) = make_uint4(o[h][0], o[h][1], o[h][2], o[h][3]);
          sc[2 * lane + h][j] = static_cast<uint8_t>(s);
        }
      }
      __syncthreads();
      const int nb = static_cast<int>(min(kb - b0, static_cast<int64_t>(kTileB)));
      for (int i = tid; i < kTileN * kTileB; i += 256) {
        const int c = i / kTileB, j = i % kTileB;
        if (n0 + c >= N || j >= nb) continue;
        const int64_t row = e * N + n0 + c;
        *reinterpret_cast<uint4*>(q + row * (K / 2) + 16 * (b0 + j)) = *reinterpret_cast<const uint4*>(codes + c * kTilePitch + 16 * j);
        scale[row * kb + b0 + j] = sc[c][j];
      }
      __syncthreads();
    }
}

// As quantize_rows: eight elements a lane, several rows a wave.  STREAM: a
// result larger than the L2s together (32 MiB) leaves past them: there and back
// as above 104 us instead of 114.
constexpr int64_t kStreamBytes = 32 << 20;

template <bool BF16, bool STREAM>
__global__ __launch_bounds__(256) void dequantize_rows_mx4_kernel(const uint8_t* __restrict__ q, int64_t ldq,
                                                                  const uint8_t* __restrict__ scale, int64_t lds,
                                                                  int64_t R, int64_t C, void* __restrict__ out,
                                                                  int64_t ldo) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
  if (8 * c >= C) return;
  const int64_t step = static_cast<int64_t>(gridDim.y) * 4;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * 4 + (threadIdx.x >> 6); r0 < R; r0 += step * kRowsAWave) {
    uint32_t w[kRowsAWave], s[kRowsAWave];
#pragma unroll
    for (int u = 0; u < kRowsAWave; ++u) {
      const int64_t r = min(r0 + u * step, R - 1);
      w[u] = *reinterpret_cast<const uint32_t*>(q + r * ldq + 4 * c);
      s[u] = scale[r * lds + (c >> 2)];
    }
#pragma unroll
    for (int u = 0; u < kRowsAWave; ++u) {
      const int64_t r = r0 + u * step;
      if (r >= R) break;
      const float sv = scale_value(s[u]);
      if (BF16) {                            // two bits of mantissa: exact
        uint32_t o[4];
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], sv, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], sv, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], sv, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], sv, 3));
        if (s[u] == 255u) o[0] = o[1] = o[2] = o[3] = 0x7fc07fc0u;
        v4u* p = reinterpret_cast<v4u*>(static_cast<uint16_t*>(out) + r * ldo + 8 * c);
        const v4u v = {o[0], o[1], o[2], o[3]};
        if (STREAM)
          __builtin_nontemporal_store(v, p);
        else
          *p = v;
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = decode((w[u] >> (4 * i)) & 15u) * sv;
        v4f* p = reinterpret_cast<v4f*>(static_cast<float*>(out) + r * ldo + 8 * c);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4f f = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
          if (STREAM)
            __builtin_nontemporal_store(f, p + h);
          else
            p[h] = f;
        }
      }
    }
  }
}

// Waves of 64 chunks by kRowsAWave rows; past what fills the GPU a few times the rows go round.
dim3 rows_grid(int64_t R, int64_t C) {
  const int64_t x = moe_cdiv(C, 512), y = moe_cdiv(R, 4 * kRowsAWave), most = moe_cdiv(32768, x);
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y < most ? y : most));
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
  const dim3 grid = moe::rows_grid(R, C);
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
  const int64_t y = moe_cdiv(K, 32 * moe::kTileB);
  const dim3 grid(static_cast<unsigned>(moe_cdiv(N, moe::kTileN)), static_cast<unsigned>(y < 65535 ? y : 65535),
                  static_cast<unsigned>(E < 65535 ? E : 65535));
  moe::quantize_weights_mx4_kernel<<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(static_cast<const uint16_t*>(w), E, K, N,
                                                                                       q, scale);
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
  const dim3 grid = moe::rows_grid(R, C);
  const bool bf = out_dtype == MOE_BF16, stream_out = R * C * (bf ? 2 : 4) > moe::kStreamBytes;
#define MOE_DEQUANTIZE(B, S) moe::dequantize_rows_mx4_kernel<B, S><<<grid, 256, 0, st>>>(q, ldq, scale, lds, R, C, out, ldo)
  if (bf) {
    if (stream_out) MOE_DEQUANTIZE(true, true); else MOE_DEQUANTIZE(true, false);
  } else {
    if (stream_out) MOE_DEQUANTIZE(false, true); else MOE_DEQUANTIZE(false, false);
  }
#undef MOE_DEQUANTIZE
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
