// moe_gmm_b128, moe_tgmm_b128: grouped products of e4m3 operands that share a
// scale over every 128 elements of the contraction, on the gfx950 scaled matrix
// cores (v_mfma_scale_f32_16x16x128_f8f6f4, float32 accumulate):
//   gmm    out[r, c] = sum_b sx[r, b] sw[g, b, c / 128] sum_{k in b} X[r, k] W_g[c, k]
//   tgmm   out[g, k, c] = sum_b sx[b, k] sy[b, c] sum_{r in b} Xt[k, r] Yt[c, r]
// One matrix instruction spans one block of the contraction, and its e8m0
// operands apply both scales: they cost nothing.  (Float32 weight scales are
// applied to each block's product as it is added, one operation an element.)
//
// An MFMA lane l supplies row l%16 of each operand, two 16-byte pieces of the
// 128: elements 16*(l/16) .. and 64 + 16*(l/16) .. (any share does, as both
// operands take the same and the scale is one for all).  The product is formed
// transposed per 16 x 16 block (the weights are the first operand), so output
// lane l holds row l%16 and four consecutive columns 4*(l/16) .. +3.
#include "b128_common.hpp"
#include "stage_common.hpp"

namespace moe {
namespace {
using namespace tile;
using namespace stage;

enum Kind { kGmmE8M0, kGmmF32, kTgmm };

struct B128Args {
  const uint8_t* x;            // gmm: rows [M, K]; tgmm: [K, cols]
  int64_t ldx;
  const uint8_t* xs;           // gmm: [M, lds]; tgmm: [cols / 128, K]
  int64_t lds;
  const uint8_t* w;            // gmm: [El, N, K]; tgmm: [N, cols]
  const void* ws;              // gmm: [El, kb, nb]; tgmm: [cols / 128, N]
  const int32_t* sizes;
  int g0, El;
  int64_t M, K, N;
  void* out;
  int32_t* err;
};

__device__ __forceinline__ v4f mfma_scaled(const v8i& w, uint32_t ws, const v8i& x, uint32_t xs, const v4f& c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, ws, 0, xs);
}

__device__ __forceinline__ v8i frag(const uint4& a, const uint4& b) {
  return v8i{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
             static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
}

template <bool OUT_BF16>
__device__ __forceinline__ void store4(void* out, int64_t at, const v4f& v) {
  if (OUT_BF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(f32_to_bf16(v[0]) | static_cast<uint32_t>(f32_to_bf16(v[1])) << 16,
                   f32_to_bf16(v[2]) | static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
  else
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
}

// ------------------------------------------------------------ 16 x 16 tiles
// A workgroup takes one tile, the contraction's blocks dealt out to its waves,
// whose sums are added in wave order.
constexpr int kSplit = 8;

struct SmallLds {
  GroupTable gt;
  int tmp[kMaxLocal];
  v4f part[kSplit][64];
};

template <Kind KIND, bool OUT_BF16>
__global__ __launch_bounds__(64 * kSplit) void b128_small_kernel(const B128Args p) {
  __shared__ SmallLds sm;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l15 = lane & 15, grp = lane >> 4;
  const int NT = static_cast<int>(p.N / 16), KT = static_cast<int>(p.K / 16);
  constexpr bool TG = KIND == kTgmm;
  // gmm: a group's row tiles by column tiles; tgmm: every group's K by N tiles (the table then counts its 128-row blocks)
  build_groups(p.sizes, p.g0, p.El, p.M, TG ? 1 : NT, TG ? b128::kBlock : 16, p.err, sm.gt, sm.tmp);
  const int64_t total = TG ? static_cast<int64_t>(p.El) * KT * NT : sm.gt.tiles_off[p.El];
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    int g, rows;
    int64_t row0, col0, wrow0;
    int kb, kend;                                  // blocks of the contraction, and its end in bytes
    const uint8_t *xp, *wp;
    int64_t ldx, ldw;
    if (TG) {
      g = static_cast<int>(t / (static_cast<int64_t>(KT) * NT));
      const int64_t l = t - static_cast<int64_t>(g) * KT * NT;
      row0 = 16 * (l / NT);
      col0 = 16 * (l % NT);
      rows = 16;
      wrow0 = col0;
      kb = sm.gt.tiles_off[g + 1] - sm.gt.tiles_off[g];
      kend = kb * 128;
      ldx = ldw = p.ldx;
      xp = p.x + static_cast<int64_t>(sm.gt.tiles_off[g]) * 128;
      wp = p.w + static_cast<int64_t>(sm.gt.tiles_off[g]) * 128;
    } else {
      g = find_group(sm.gt, p.El, static_cast<int>(t));
      const int m = sm.gt.rows_off[g + 1] - sm.gt.rows_off[g], l = static_cast<int>(t) - sm.gt.tiles_off[g], nr = (m + 15) / 16;
      row0 = sm.gt.rows_off[g] + 16 * (l % nr);
      rows = min(16, m - 16 * (l % nr));
      col0 = 16 * (l / nr);
      wrow0 = static_cast<int64_t>(g) * p.N + col0;
      kend = static_cast<int>(p.K);
      kb = (kend + 127) / 128;
      ldx = p.ldx;
      ldw = p.K;
      xp = p.x;
      wp = p.w;
    }
    const int64_t xrow = row0 + min(l15, rows - 1);
    const uint8_t* xa = xp + xrow * ldx;
    const uint8_t* wa = wp + (wrow0 + l15) * ldw;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    const int per = (kb + kSplit - 1) / kSplit;
    for (int b = wave * per; b < min(kb, (wave + 1) * per); ++b) {
      uint4 xv[2], wv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = 128 * b + 64 * h + 16 * grp;
        xv[h] = wv[h] = make_uint4(0, 0, 0, 0);
        if (at < kend) {
          xv[h] = *reinterpret_cast<const uint4*>(xa + at);
          wv[h] = *reinterpret_cast<const uint4*>(wa + at);
        }
      }
      if constexpr (TG) {
        const int64_t blk = sm.gt.tiles_off[g] + b;
        acc = mfma_scaled(frag(wv[0], wv[1]), static_cast<const uint8_t*>(p.ws)[blk * p.N + wrow0 + l15], frag(xv[0], xv[1]),
                          p.xs[blk * p.K + xrow], acc);
      } else {
        const int64_t nb = (p.N + 127) / 128, at = (static_cast<int64_t>(g) * kb + b) * nb + col0 / 128;
        const uint32_t xs = p.xs[xrow * p.lds + b];
        if constexpr (KIND == kGmmE8M0)
          acc = mfma_scaled(frag(wv[0], wv[1]), static_cast<const uint8_t*>(p.ws)[at], frag(xv[0], xv[1]), xs, acc);
        else
          acc += static_cast<const float*>(p.ws)[at] * mfma_scaled(frag(wv[0], wv[1]), 127, frag(xv[0], xv[1]), xs, v4f{0.f, 0.f, 0.f, 0.f});
      }
    }
    __syncthreads();
    sm.part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      acc = sm.part[0][lane];
#pragma unroll
      for (int i = 1; i < kSplit; ++i) acc += sm.part[i][lane];
      if (l15 < rows)
        store4<OUT_BF16>(p.out, (TG ? static_cast<int64_t>(g) * p.K + row0 + l15 : row0 + l15) * p.N + col0 + 4 * grp, acc);
    }
  }
  if constexpr (!TG) {                             // rows past the last group's are zero
    const int64_t n_rows = sm.gt.rows_off[p.El], bytes = (p.M - n_rows) * p.N * (OUT_BF16 ? 2 : 4);
    uint8_t* z = static_cast<uint8_t*>(p.out) + n_rows * p.N * (OUT_BF16 ? 2 : 4);
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 64 * kSplit + tid) * 16; i < bytes; i += static_cast<int64_t>(gridDim.x) * 64 * kSplit * 16)
      *reinterpret_cast<uint4*>(z + i) = make_uint4(0, 0, 0, 0);
  }
}

template <Kind KIND, bool OUT_BF16>
hipError_t launch_b128(const B128Args& p, hipStream_t st) {
  b128_small_kernel<KIND, OUT_BF16><<<4 * num_cus(), 64 * kSplit, 0, st>>>(p);
  return hipGetLastError();
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

size_t gmm_b128_ws_bytes() { return tile::kHdr; }
size_t tgmm_b128_ws_bytes() { return tile::kHdr; }

}  // namespace moe

extern "C" int moe_gmm_b128(const uint8_t* lhs, int64_t ldl, const uint8_t* lhs_scale, int64_t lds, const uint8_t* rhs,
                            const void* rhs_scale, int rhs_scale_dtype, const int32_t* group_sizes, int32_t E,
                            int32_t group_offset, int32_t num_local_experts, int64_t M, int64_t K, int64_t N, int out_dtype,
                            void* out, void* ws, size_t ws_bytes, void* stream) {
  using moe::tile::kMaxLocal;
  if (M < 0 || K <= 0 || N <= 0 || K % 16 || N % 16) return MOE_ERR_SHAPE;
  if (E <= 0 || E > 1024 || group_offset < 0 || num_local_experts < 0 || num_local_experts > kMaxLocal ||
      group_offset > E - num_local_experts)
    return MOE_ERR_SHAPE;
  // row offsets inside a tile, and a group's weights' scales, are 32-bit
  if (M > INT32_MAX - 1 || K > (1 << 22) || ldl > (1 << 23) || N > INT32_MAX || N * moe_cdiv(K, 128) > INT32_MAX) return MOE_ERR_SHAPE;
  // the tile table of any split of M rows into the groups stays below 2^31 entries
  if ((moe_cdiv(M, 16) + num_local_experts + 1) * (N / 16) > INT32_MAX) return MOE_ERR_SHAPE;
  if (ldl < K || ldl % 16 || lds < moe_cdiv(K, 128) || lds % 16 || lds > (1 << 23)) return MOE_ERR_SHAPE;
  if (rhs_scale_dtype != MOE_E8M0 && rhs_scale_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (out_dtype == MOE_DTYPE_DEFAULT || out_dtype == MOE_E4M3FN) out_dtype = MOE_BF16;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!out || !group_sizes) return MOE_ERR_NULL;
  if (num_local_experts > 0 && (!lhs || !lhs_scale || !rhs || !rhs_scale)) return MOE_ERR_NULL;
  if (!moe::aligned16(lhs) || !moe::aligned16(lhs_scale) || !moe::aligned16(rhs) || !moe::aligned16(out) ||
      (rhs_scale_dtype == MOE_F32 && reinterpret_cast<uintptr_t>(rhs_scale) % 4))
    return MOE_ERR_SHAPE;
  if (!ws || ws_bytes < moe::gmm_b128_ws_bytes()) return MOE_ERR_WORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const moe::B128Args p{lhs, ldl, lhs_scale, lds, rhs, rhs_scale, group_sizes, group_offset, num_local_experts, M, K, N, out,
                        static_cast<int32_t*>(ws)};
  const bool bf = out_dtype == MOE_BF16;
  hipError_t e;
  if (rhs_scale_dtype == MOE_E8M0)
    e = bf ? moe::launch_b128<moe::kGmmE8M0, true>(p, st) : moe::launch_b128<moe::kGmmE8M0, false>(p, st);
  else
    e = bf ? moe::launch_b128<moe::kGmmF32, true>(p, st) : moe::launch_b128<moe::kGmmF32, false>(p, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

extern "C" int moe_tgmm_b128(const uint8_t* lhs_t, const uint8_t* lhs_scale, const uint8_t* rhs_t, const uint8_t* rhs_scale,
                             const int32_t* group_sizes, int32_t E, int32_t group_offset, int32_t num_local_experts, int64_t M,
                             int64_t K, int64_t N, int out_dtype, void* out, void* ws, size_t ws_bytes, void* stream) {
  using moe::tile::kMaxLocal;
  if (M < 0 || K <= 0 || N <= 0 || K % 16 || N % 16 || K > INT32_MAX || N > INT32_MAX) return MOE_ERR_SHAPE;
  if (E <= 0 || E > 1024 || group_offset < 0 || num_local_experts < 0 || num_local_experts > kMaxLocal ||
      group_offset > E - num_local_experts)
    return MOE_ERR_SHAPE;
  if (M > (int64_t{1} << 24) || M + 128 * static_cast<int64_t>(E) > (int64_t{1} << 24)) return MOE_ERR_SHAPE;
  // tiles are counted in 32 bits
  if (moe_cdiv(K, 16) * moe_cdiv(N, 16) > INT32_MAX / (num_local_experts > 0 ? num_local_experts : 1)) return MOE_ERR_SHAPE;
  if (out_dtype == MOE_DTYPE_DEFAULT) out_dtype = MOE_F32;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (num_local_experts == 0) return MOE_OK;
  if (!out || !group_sizes) return MOE_ERR_NULL;
  if (M > 0 && (!lhs_t || !lhs_scale || !rhs_t || !rhs_scale)) return MOE_ERR_NULL;
  if (!moe::aligned16(lhs_t) || !moe::aligned16(lhs_scale) || !moe::aligned16(rhs_t) || !moe::aligned16(rhs_scale) ||
      !moe::aligned16(out))
    return MOE_ERR_SHAPE;
  if (!ws || ws_bytes < moe::tgmm_b128_ws_bytes()) return MOE_ERR_WORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  int64_t cols = 0;
  if (moe_tgmm_xt_cols(M, E, &cols) != MOE_OK) return MOE_ERR_SHAPE;
  const moe::B128Args p{lhs_t, cols, lhs_scale, 0, rhs_t, rhs_scale, group_sizes, group_offset, num_local_experts, M, K, N, out,
                        static_cast<int32_t*>(ws)};
  const hipError_t e = out_dtype == MOE_BF16 ? moe::launch_b128<moe::kTgmm, true>(p, st) : moe::launch_b128<moe::kTgmm, false>(p, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
