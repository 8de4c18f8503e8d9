// moe_quantize_rows_b128, moe_quantize_weights_b128, moe_quantize_cols_b128:
// to e4m3 with a power-of-two scale for every block of 128 along a row, of 128
// by 128, and of 128 along a group's rows (b128_common.hpp).  v / scale is exact,
// the scale a power of two, so a code is v's nearest with one rounding.  Memory
// bounds all three: 2 bytes in, 1 out (2 for weights in both orientations).
// Measured: rows of 8192 x 7168 31 us (5.7 TB/s), gated 62 to 74 (4.0 to 4.7); weights of
// 8 x 7168 x 2048 96 us (4.9 TB/s); columns of 32768 x 1536 51 us (3.0 TB/s; 30 where the
// rows lie in the caches), gated 73 (3.4), of 32768 x 4096 gathered from 8192 tokens 80 us
// (2.5 TB/s of the bytes that leave the caches).
#include "b128_common.hpp"
#include "quant_common.hpp"

namespace moe {
namespace {
using namespace b128;

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// Read once here, and not kept in the caches.
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p)));
}

template <bool SILU>
__device__ __forceinline__ void values8(const uint4& a, const uint4& b, float (&v)[8]) {
  const Bf16x8 av{a};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = av.get(i);
  if constexpr (SILU) {
    const Bf16x8 bv{b};
    float g[8], h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { g[i] = v[i]; h[i] = bv.get(i); }
    silu_mul8(g, h, v);
  }
}

__device__ __forceinline__ uint32_t max_lane(uint32_t v, uint32_t o) { return v > o ? v : o; }
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xf, 0xf, true));
}

// Sixteen lanes hold one block, eight elements each; a wave takes 64 such
// chunks of kRowsAWave rows, its loads first.
constexpr int kRowsAWave = 4;

template <bool SILU>
__global__ __launch_bounds__(256) void quantize_rows_b128_kernel(const uint16_t* __restrict__ x,
                                                                 const uint16_t* __restrict__ x_up, int64_t ldx, int64_t R,
                                                                 int64_t C, uint8_t* __restrict__ q, int64_t ldq,
                                                                 uint8_t* __restrict__ scale, int64_t lds) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
  const bool in = 8 * c < C;                 // (lanes past the row stay for the block's maximum)
  const int64_t step = static_cast<int64_t>(gridDim.y) * 4;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * 4 + (threadIdx.x >> 6); r0 < R; r0 += step * kRowsAWave) {
    uint4 a[kRowsAWave], b[SILU ? kRowsAWave : 1];
#pragma unroll
    for (int u = 0; u < kRowsAWave; ++u) {
      const int64_t r = min(r0 + u * step, R - 1);
      a[u] = make_uint4(0, 0, 0, 0);
      if (in) a[u] = load_once(x + r * ldx + 8 * c);
      if constexpr (SILU) {
        b[u] = make_uint4(0, 0, 0, 0);
        if (in) b[u] = load_once(x_up + r * ldx + 8 * c);
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsAWave; ++u) {
      const int64_t r = r0 + u * step;
      if (r >= R) break;
      float v[8];
      values8<SILU>(a[u], b[SILU ? u : 0], v);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
      top = max_lane(top, moved<0xB1>(top));           // lane ^ 1, ^ 2, then halves and rows of 16 mirrored
      top = max_lane(top, moved<0x4E>(top));
      top = max_lane(top, moved<0x141>(top));
      top = max_lane(top, moved<0x140>(top));
      const uint32_t s = scale_code(top);
      if (in) {
        *reinterpret_cast<uint2*>(q + r * ldq + 8 * c) = encode8(v, inverse(s));
        if ((c & 15) == 0) scale[r * lds + (c >> 4)] = static_cast<uint8_t>(s);
      }
    }
  }
}

// 128 x 128 codes in LDS, one column of the input a row of it.
constexpr int kPitch = kBlock + 16;

// Eight rows of eight bytes (a row an uint2) to eight columns of eight.
__device__ __forceinline__ void transpose8(const uint2 (&r)[8], uint2 (&c)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {            // columns 4 h .. of rows 4 k .. : a 4 x 4 block
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = h ? r[4 * k + i].y : r[4 * k + i].x;
      const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
      const uint32_t d = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), e = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
      const uint32_t o[4] = {__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(b, a, 0x07060302u),
                             __builtin_amdgcn_perm(e, d, 0x05040100u), __builtin_amdgcn_perm(e, d, 0x07060302u)};
#pragma unroll
      for (int i = 0; i < 4; ++i) (k ? c[4 * h + i].y : c[4 * h + i].x) = o[i];
    }
  }
}

// A workgroup takes one block of 128 by 128.  A thread holds eight rows of
// eight columns; the codes of the transposed orientation go through LDS, so
// that both leave as whole lines.
__global__ __launch_bounds__(256) void quantize_weights_b128_kernel(const uint16_t* __restrict__ w, int64_t E, int64_t K,
                                                                    int64_t N, uint8_t* __restrict__ q,
                                                                    uint8_t* __restrict__ scale, uint8_t* __restrict__ qt,
                                                                    uint8_t* __restrict__ scale_t) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[kBlock * kPitch];
  __shared__ uint32_t red[4];
  const int64_t nb = (N + kBlock - 1) / kBlock, kb = (K + kBlock - 1) / kBlock;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kBlock;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t n = n0 + 8 * tx;
  for (int64_t e = blockIdx.z; e < E; e += gridDim.z)
    for (int64_t b = blockIdx.y; b < kb; b += gridDim.y) {
      const int64_t k0 = b * kBlock + 8 * ty;
      const bool in = n < N && k0 < K;       // (K and N are multiples of 16: all of a thread's rows and columns exist, or none)
      uint4 a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = make_uint4(0, 0, 0, 0);
        if (in) a[i] = load_once(w + (e * K + k0 + i) * N + n);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t p[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max((p[j] << 16) & 0x7fffffffu, p[j] & 0x7fff0000u));
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o, 64)));
      if ((tid & 63) == 0) red[tid >> 6] = top;
      __syncthreads();
      const uint32_t s = scale_code(max(max(red[0], red[1]), max(red[2], red[3])));
      const float inv = inverse(s);
      uint2 r[8], c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v[8];
        values8<false>(a[i], a[i], v);
        r[i] = encode8(v, inv);
        if (qt && in) *reinterpret_cast<uint2*>(qt + (e * K + k0 + i) * N + n) = r[i];
      }
      if (q) {
        transpose8(r, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) *reinterpret_cast<uint2*>(codes + (8 * tx + j) * kPitch + 8 * ty) = c[j];
      }
      if (tid == 0) {
        if (scale) scale[(e * kb + b) * nb + blockIdx.x] = static_cast<uint8_t>(s);
        if (scale_t) scale_t[(e * nb + blockIdx.x) * kb + b] = static_cast<uint8_t>(s);
      }
      __syncthreads();
      if (q) {
        const int64_t kc = b * kBlock + 16 * (tid & 7);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (tid >> 3) + 32 * i;
          if (n0 + row < N && kc < K)
            *reinterpret_cast<uint4*>(q + (e * N + n0 + row) * K + kc) =
                *reinterpret_cast<const uint4*>(codes + row * kPitch + 16 * (tid & 7));
        }
      }
    }
}

struct ColsArgs {
  const uint16_t *x, *x_up;
  int64_t ldx, T;
  int k;
  const int32_t* perm;
  const int32_t* sizes;
  int g0, El;
  int64_t M, C;
  uint8_t* qt;
  uint8_t* scale;
  int32_t* err;
};

// A workgroup takes 128 rows of one group and every gridDim.y-th 128 of the
// columns, the next ones' loads issued before these are worked on.  A thread
// holds eight rows of eight columns; a column's maximum goes through LDS, and so
// do its codes, which leave as lines of 128 bytes, one run for all columns.
template <bool SILU>
__global__ __launch_bounds__(256) void quantize_cols_b128_kernel(const ColsArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[kBlock * kPitch];
  __shared__ uint32_t tops[16][kBlock + 4];
  __shared__ float invs[kBlock];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int blk = blockIdx.x;
  if (blk == 0 && blockIdx.y == 0 && tid < 64)
    find_block(p.sizes + p.g0, p.El, static_cast<int>(p.M), INT32_MAX, p.err);    // (a pass over every group, for what is wrong)
  const GroupBlock f = find_block(p.sizes + p.g0, p.El, static_cast<int>(p.M), blk, nullptr);
  if (f.g < 0) return;
  const int r0 = (blk - f.block0) * kBlock + 8 * ty;                     // first of the thread's rows in its group
  const uint16_t *xr[8], *ur[SILU ? 8 : 1];
  int64_t start = 0;                         // the window's first slot
  if (p.perm) {
    for (int g = tid & 63; g < p.g0; g += 64) start += max(p.sizes[g], 0);
    if (p.g0 > 0)
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) start += __shfl_xor(start, o, 64);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int64_t row = f.row0 + min(r0 + i, f.m - 1);
    if (p.perm) row = min(static_cast<int64_t>(max(p.perm[min(start + row, p.T * p.k - 1)], 0)) / p.k, p.T - 1);
    xr[i] = p.x + row * p.ldx + 8 * tx;
    if constexpr (SILU) ur[i] = p.x_up + row * p.ldx + 8 * tx;
  }
  uint4 a[8], b[SILU ? 8 : 1];
  const int step = gridDim.y * kBlock;
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = r0 + i < f.m && c0 + 8 * tx < p.C;
      a[i] = make_uint4(0, 0, 0, 0);
      if (in) a[i] = *reinterpret_cast<const uint4*>(xr[i] + c0);
      if constexpr (SILU) {
        b[i] = make_uint4(0, 0, 0, 0);
        if (in) b[i] = *reinterpret_cast<const uint4*>(ur[i] + c0);
      }
    }
  };
  int c0 = blockIdx.y * kBlock;
  if (c0 < p.C) load(c0);
  for (; c0 < p.C; c0 += step) {
    uint32_t top[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    uint4 raw[8];                            // (plain rows stay as they came: half the registers)
    float v[SILU ? 8 : 1][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      raw[i] = a[i];
      if constexpr (SILU) values8<true>(a[i], b[i], v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) top[j] = max(top[j], magnitude(SILU ? v[SILU ? i : 0][j] : Bf16x8{a[i]}.get(j)));
    }
    if (c0 + step < p.C) load(c0 + step);
#pragma unroll
    for (int j = 0; j < 8; j += 4) *reinterpret_cast<uint4*>(&tops[ty][8 * tx + j]) = make_uint4(top[j], top[j + 1], top[j + 2], top[j + 3]);
    __syncthreads();
    if (tid < kBlock) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) t = max(t, tops[i][tid]);
      const uint32_t s = scale_code(t);
      invs[tid] = inverse(s);
      if (c0 + tid < p.C) p.scale[blk * p.C + c0 + tid] = static_cast<uint8_t>(s);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = SILU ? v[SILU ? i : 0][j] : Bf16x8{raw[i]}.get(j);
      *reinterpret_cast<uint2*>(codes + (8 * tx + j) * kPitch + 8 * ty) = encode8(u, invs[8 * tx + j]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = (tid >> 3) + 32 * i;
      if (c0 + col < p.C)
        *reinterpret_cast<uint4*>(p.qt + (blk * p.C + c0 + col) * kBlock + 16 * (tid & 7)) =
            *reinterpret_cast<const uint4*>(codes + col * kPitch + 16 * (tid & 7));
    }
    // (the next columns' maxima touch `tops` alone until their first barrier, behind these reads)
  }
}

dim3 rows_grid(int64_t R, int64_t C) {
  const int64_t x = moe_cdiv(C, 512), y = moe_cdiv(R, 4 * kRowsAWave), most = moe_cdiv(32768, x);
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y < most ? y : most));
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace moe

extern "C" int moe_quantize_rows_b128(const void* x, const void* x_up, int64_t ldx, int act, int64_t R, int64_t C,
                                      uint8_t* q, int64_t ldq, uint8_t* scale, int64_t lds, void* stream) {
  if (R < 0 || C <= 0 || C % 16 || C > INT32_MAX || ldx < C || ldx % 8 || ldq < C || ldq % 16 || lds < moe_cdiv(C, 128)) return MOE_ERR_SHAPE;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SILU_MUL) return MOE_ERR_UNSUPPORTED;
  if (act == MOE_ACT_NONE && x_up) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!x || !q || !scale || (act == MOE_ACT_SILU_MUL && !x_up)) return MOE_ERR_NULL;
  if (!moe::aligned(x, 16) || !moe::aligned(x_up, 16) || !moe::aligned(q, 16)) return MOE_ERR_SHAPE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const uint16_t *xa = static_cast<const uint16_t*>(x), *xb = static_cast<const uint16_t*>(x_up);
  const dim3 grid = moe::rows_grid(R, C);
  if (act == MOE_ACT_SILU_MUL)
    moe::quantize_rows_b128_kernel<true><<<grid, 256, 0, st>>>(xa, xb, ldx, R, C, q, ldq, scale, lds);
  else
    moe::quantize_rows_b128_kernel<false><<<grid, 256, 0, st>>>(xa, xb, ldx, R, C, q, ldq, scale, lds);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_quantize_weights_b128(const void* w, int64_t E, int64_t K, int64_t N, uint8_t* q, uint8_t* scale,
                                         uint8_t* qt, uint8_t* scale_t, void* stream) {
  if (E < 0 || K <= 0 || K % 16 || N <= 0 || N % 16) return MOE_ERR_SHAPE;
  if (E == 0) return MOE_OK;
  if (!w || (!q && !qt) || !q != !scale || !qt != !scale_t) return MOE_ERR_NULL;
  if (!moe::aligned(w, 16) || !moe::aligned(q, 16) || !moe::aligned(qt, 16)) return MOE_ERR_SHAPE;
  const int64_t x = moe_cdiv(N, moe::kBlock), y = moe_cdiv(K, moe::kBlock);
  if (x > (1 << 23)) return MOE_ERR_SHAPE;        // (threads of a launch in one dimension: below 2^32)
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y < 4096 ? y : 4096), static_cast<unsigned>(E < 1024 ? E : 1024));
  moe::quantize_weights_b128_kernel<<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(static_cast<const uint16_t*>(w), E, K, N,
                                                                                        q, scale, qt, scale_t);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_quantize_cols_b128(const void* x, const void* x_up, int64_t ldx, int act, int64_t T, int32_t k,
                                      const int32_t* perm, const int32_t* group_sizes, int32_t E, int32_t group_offset,
                                      int32_t num_local_experts, int64_t M, int64_t C, uint8_t* qt, uint8_t* scale_t, void* ws,
                                      size_t ws_bytes, void* stream) {
  if (M < 0 || C <= 0 || C % 16 || C > INT32_MAX || ldx < C || ldx % 8 || T < 0 || k < 1 || k > 64) return MOE_ERR_SHAPE;
  if (E <= 0 || E > 1024 || group_offset < 0 || num_local_experts < 0 || group_offset > E - num_local_experts) return MOE_ERR_SHAPE;
  if (M > (int64_t{1} << 23) || M + 128 * static_cast<int64_t>(E) > (int64_t{1} << 23)) return MOE_ERR_SHAPE;
  if (T > INT32_MAX || (!perm && T < M)) return MOE_ERR_SHAPE;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SILU_MUL) return MOE_ERR_UNSUPPORTED;
  if (act == MOE_ACT_NONE && x_up) return MOE_ERR_UNSUPPORTED;
  if (M == 0 || num_local_experts == 0 || T == 0) return MOE_OK;
  if (!x || !group_sizes || !qt || !scale_t || (act == MOE_ACT_SILU_MUL && !x_up)) return MOE_ERR_NULL;
  if (!moe::aligned(x, 16) || !moe::aligned(x_up, 16) || !moe::aligned(qt, 16) || !moe::aligned(scale_t, 16)) return MOE_ERR_SHAPE;
  if (!ws || ws_bytes < 256) return MOE_ERR_WORKSPACE;
  const moe::ColsArgs p{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(x_up), ldx, T, k, perm, group_sizes,
                        group_offset, num_local_experts, M, C, qt, scale_t, static_cast<int32_t*>(ws)};
  // as many blocks as any split of M rows into the groups has
  const int64_t groups = num_local_experts < M ? num_local_experts : M;
  const int64_t blocks = moe_cdiv(M, 128) + groups, tiles = moe_cdiv(C, 128);
  const int64_t y = moe_cdiv(2560, blocks) < tiles ? moe_cdiv(2560, blocks) : tiles;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(y));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (act == MOE_ACT_SILU_MUL)
    moe::quantize_cols_b128_kernel<true><<<grid, 256, 0, st>>>(p);
  else
    moe::quantize_cols_b128_kernel<false><<<grid, 256, 0, st>>>(p);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
