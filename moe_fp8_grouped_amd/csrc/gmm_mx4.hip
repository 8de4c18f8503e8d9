// moe_gmm_mx4: grouped matmul with 4-bit block-scaled weights on the gfx950
// scaled matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4, float32
// accumulate):
//   out[r, c] = ls[r] * sum_k X[r, k] W_g[k, c]
// for the rows r of local group g, W e2m1 codes with one e8m0 scale for every
// 32 along k, X e4m3fn with a float scale a row (or one for all), or in the
// weights' own format (then there is no ls).
//
// An MFMA lane l supplies row l%16 of each operand.  Of a 4-bit operand it
// holds the contraction elements 32*(l/16) .. +31 and their scale byte: one
// block of the format is one lane's share.  Of an e4m3 operand it holds two
// 16-byte pieces, elements 16*(l/16) .. +15 and 64 + 16*(l/16) .. +15 (both
// layouts measured on the device, one element at a time).  The product is
// formed transposed per 16 x 16 block (the weights are the first operand), so
// output lane l holds row l%16 and four consecutive columns 4*(l/16) .. +3.
#include "mx4_common.hpp"
#include "tile_common.hpp"

namespace moe {
namespace {
using namespace tile;

// First operand e2m1 (format 4); second e4m3 (0) or e2m1 (4).
template <bool A8>
__device__ __forceinline__ v4f mfma_mx4(const v8i& w, uint32_t ws, const v8i& x, uint32_t xs, const v4f& c) {
  if constexpr (A8)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, 0, 0, ws, 0, xs);
  else
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, 4, 0, ws, 0, xs);
}

__device__ __forceinline__ v8i frag16(uint4 a) {
  return v8i{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
}

struct Mx4Args {
  const uint8_t* lhs;
  int64_t ldl;                 // bytes a lhs row
  const void* ls;              // A8: float [M] or [1]; else e8m0 rows
  int64_t lds;                 // bytes a row of lhs scales (not A8)
  int ls_per_row;
  const uint8_t* rhs;          // [El, N, K/2]
  const uint8_t* rs;           // [El, N, K/32]
  const int32_t* group_sizes;
  int g0, El;
  int64_t M, K, N;
  void* out;
  int32_t* err;
};

constexpr int E_BM = 64, E_BN = 64;

// Any K (a multiple of 32) and N (of 16): 64 x 64 tiles, a wave 16 rows x 64
// columns, operands from global memory into registers.
template <bool A8, bool OUT_BF16>
__global__ __launch_bounds__(256) void gmm_mx4_edge_kernel(const Mx4Args p) {
  __shared__ GroupTable gt;
  __shared__ int tmp[kMaxLocal];
  const int NT = static_cast<int>((p.N + E_BN - 1) / E_BN);
  build_groups(p.group_sizes, p.g0, p.El, p.M, NT, E_BM, p.err, gt, tmp);
  const int total = gt.tiles_off[p.El];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l15 = lane & 15, grp = lane >> 4;
  const int64_t K = p.K, N = p.N, kb = K / 32;
  const int steps = static_cast<int>((kb + 3) / 4);
  int first, last, step;
  xcd_share(total, first, last, step);
  for (int t = first; t < last; t += step) {
    const int g = find_group(gt, p.El, t);
    const int local = t - gt.tiles_off[g];
    const int m_g = gt.rows_off[g + 1] - gt.rows_off[g];
    const int mt = (m_g + E_BM - 1) / E_BM;
    const int nt = local / mt;
    const int roff = (local - nt * mt) * E_BM + wave * 16;      // this wave's first row in the group
    if (roff >= m_g) continue;
    const int64_t row = gt.rows_off[g] + min(roff + l15, m_g - 1);
    const int64_t col0 = static_cast<int64_t>(nt) * E_BN;
    const uint8_t* xrow = p.lhs + row * p.ldl;
    v4f acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < steps; ++s) {
      const int64_t b = 4 * s + grp;          // this lane's block
      const bool in = b < kb;
      v8i x = v8i{0, 0, 0, 0, 0, 0, 0, 0};
      uint32_t xs = 127;
      if (A8) {
        const int64_t k = 128 * static_cast<int64_t>(s) + 16 * grp;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = make_uint4(0, 0, 0, 0);
        if (k < K) lo = *reinterpret_cast<const uint4*>(xrow + k);
        if (k + 64 < K) hi = *reinterpret_cast<const uint4*>(xrow + k + 64);
        x = v8i{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
                static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
      } else if (in) {
        x = frag16(*reinterpret_cast<const uint4*>(xrow + 16 * b));
        xs = static_cast<const uint8_t*>(p.ls)[row * p.lds + b];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = min(col0 + 16 * j + l15, N - 1);
        const int64_t wr = static_cast<int64_t>(g) * N + n;
        v8i w = v8i{0, 0, 0, 0, 0, 0, 0, 0};
        uint32_t ws = 127;
        if (in) {
          w = frag16(*reinterpret_cast<const uint4*>(p.rhs + wr * (K / 2) + 16 * b));
          ws = p.rs[wr * kb + b];
        }
        acc[j] = mfma_mx4<A8>(w, ws, x, xs, acc[j]);
      }
    }
    if (roff + l15 >= m_g) continue;
    float lsr = 1.0f;
    if (A8) lsr = static_cast<const float*>(p.ls)[p.ls_per_row ? row : 0];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = col0 + 16 * j + 4 * grp;                // N is a multiple of 16: all four columns or none
      if (c >= N) continue;
      const float o[4] = {acc[j][0] * lsr, acc[j][1] * lsr, acc[j][2] * lsr, acc[j][3] * lsr};
      if (OUT_BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * N + c) =
            make_uint2(f32_to_bf16(o[0]) | (static_cast<uint32_t>(f32_to_bf16(o[1])) << 16),
                       f32_to_bf16(o[2]) | (static_cast<uint32_t>(f32_to_bf16(o[3])) << 16));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * N + c) = make_float4(o[0], o[1], o[2], o[3]);
    }
  }
  // rows past the last group's are zero
  const int64_t n_rows = gt.rows_off[p.El];
  const int64_t bytes = (p.M - n_rows) * N * (OUT_BF16 ? 2 : 4);
  uint8_t* z = static_cast<uint8_t*>(p.out) + n_rows * N * (OUT_BF16 ? 2 : 4);
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 16; i < bytes;
       i += static_cast<int64_t>(gridDim.x) * 256 * 16)
    *reinterpret_cast<uint4*>(z + i) = make_uint4(0, 0, 0, 0);
}

template <bool A8>
hipError_t launch_edge(const Mx4Args& p, bool bf16, hipStream_t st) {
  const int64_t tiles = (moe_cdiv(p.M, E_BM) + p.El) * moe_cdiv(p.N, E_BN);
  int64_t grid = 4 * num_cus();
  if (tiles < grid) grid = tiles;
  if (grid < 8) grid = 8;                     // the XCD split gives each of the 8 parts its own workgroups
  if (bf16)
    gmm_mx4_edge_kernel<A8, true><<<static_cast<unsigned>(grid), 256, 0, st>>>(p);
  else
    gmm_mx4_edge_kernel<A8, false><<<static_cast<unsigned>(grid), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t gmm_mx4_ws_bytes() { return static_cast<size_t>(tile::kHdr); }

}  // namespace moe

extern "C" int moe_gmm_mx4(const uint8_t* lhs, int64_t ldl, const void* lhs_scale, int64_t lds, int lhs_format,
                           int lhs_scale_mode, const uint8_t* rhs, const uint8_t* rhs_scale, const int32_t* group_sizes,
                           int32_t E, int32_t group_offset, int32_t num_local_experts, int64_t M, int64_t K, int64_t N,
                           int out_dtype, void* out, void* ws, size_t ws_bytes, void* stream) {
  using moe::tile::kMaxLocal;
  if (M < 0 || K <= 0 || N <= 0 || K % 32 || N % 16) return MOE_ERR_SHAPE;
  if (E <= 0 || E > 1024 || group_offset < 0 || num_local_experts < 0 || num_local_experts > kMaxLocal ||
      group_offset + num_local_experts > E)
    return MOE_ERR_SHAPE;
  if (M > INT32_MAX - 1) return MOE_ERR_SHAPE;
  // the tile table of any split of M rows into the groups stays below 2^31 entries
  if ((moe_cdiv(M, 16) + num_local_experts + 1) * moe_cdiv(N, 64) > INT32_MAX) return MOE_ERR_SHAPE;
  if (lhs_format != MOE_E4M3FN && lhs_format != MOE_MX4) return MOE_ERR_UNSUPPORTED;
  const bool a8 = lhs_format == MOE_E4M3FN;
  if (lhs_scale_mode != MOE_SCALE_ROW_DYNAMIC &&
      (!a8 || (lhs_scale_mode != MOE_SCALE_TENSOR_DYNAMIC && lhs_scale_mode != MOE_SCALE_TENSOR_STATIC)))
    return MOE_ERR_UNSUPPORTED;
  if (ldl < (a8 ? K : K / 2) || ldl % 16 || (a8 ? lds != 0 : lds < K / 32)) return MOE_ERR_SHAPE;
  if (out_dtype == MOE_DTYPE_DEFAULT || out_dtype == MOE_E4M3FN) out_dtype = MOE_BF16;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!out || !group_sizes) return MOE_ERR_NULL;
  if (num_local_experts > 0 && (!lhs || !lhs_scale || !rhs || !rhs_scale)) return MOE_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(lhs) % 16 || reinterpret_cast<uintptr_t>(rhs) % 16 ||
      reinterpret_cast<uintptr_t>(out) % 16)
    return MOE_ERR_SHAPE;
  if (!ws || ws_bytes < static_cast<size_t>(moe::tile::kHdr)) return MOE_ERR_WORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool bf16 = out_dtype == MOE_BF16;
  const moe::Mx4Args p{lhs, ldl, lhs_scale, lds, lhs_scale_mode == MOE_SCALE_ROW_DYNAMIC ? 1 : 0, rhs, rhs_scale,
                       group_sizes, group_offset, num_local_experts, M, K, N, out, static_cast<int32_t*>(ws)};
  const hipError_t e = a8 ? moe::launch_edge<true>(p, bf16, st) : moe::launch_edge<false>(p, bf16, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
