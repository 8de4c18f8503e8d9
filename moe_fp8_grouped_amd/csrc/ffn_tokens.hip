// moe_ffn_tokens: a whole gated expert layer for a few tokens,
//   out[t] = sum_j w[t, j] * ((silu(x[t] W0_e) * (x[t] W1_e)) Wo_e),  e = ids[t, j],
// in two kernels.  At these sizes the experts' weights are the traffic: each
// chosen expert's weights are read once, from e4m3 codes or 4-bit blocks
// straight into registers and converted there, while the activations stay as
// they are (bfloat16 rows; the hidden values as two bfloat16 pieces, 16 bits
// of mantissa, since they are small next to the weights) -- nothing is
// quantized, so a token's result does not depend on the others'.
//
// Both kernels form weights (16 output channels) times rows (16 slots) with
// v_mfma_f32_16x16x32_bf16; a lane holds 16 bytes of one channel's codes.
// The four waves of a workgroup split the contraction, and add up in LDS.
//   1  a, b -> h = silu(a) * b for 16 hidden channels of one expert
//   2  y[slot] for 32 output channels of one expert, to the workspace; the
//      workgroup that finishes a column block last adds each token's slots in
//      slot order and writes the output
#include "mx4_common.hpp"
#include "tile_common.hpp"

namespace moe {
namespace {
using tile::v4f;

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kMaxT = 64, kMaxSlots = 1024, kMaxLocalE = 1024;
constexpr int kThreads = 256, kWaves = 4;
constexpr int kHeader = 256;                       // workspace: error word, then the counters of the column blocks

struct FfnArgs {
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;
  const float* tw;
  int T, k;
  int64_t H, I;
  int E, g0, El;
  const uint8_t* w01;
  const void* s01;
  int kb01, nb01;
  const uint8_t* wo;
  const void* so;
  int kbo, nbo;
  void* out;
  int out_bf16;
  int32_t* err;
  int32_t* cnt;
  uint16_t* h;                                     // [2][slots][I]: high and low pieces
  float* y;                                        // [slots][H]
};

// Which local experts are met, in order, from the routing; every workgroup
// derives it for itself.
struct Routing {
  int local[kMaxSlots];                            // local expert of a slot, or -1
  int count[kMaxLocalE];
  int met[kMaxSlots];                              // the met experts, ascending
  int n_met;
};

__device__ void read_routing(const FfnArgs& p, Routing& r) {
  const int tid = threadIdx.x, n = p.T * p.k;
  for (int e = tid; e < p.El; e += kThreads) r.count[e] = 0;
  __syncthreads();
  for (int s = tid; s < n; s += kThreads) {
    const int id = p.ids[s];
    if ((id < 0 || id >= p.E) && blockIdx.x == 0) raise_error(p.err, MOE_DEVERR_EXPERT_ID);
    const int e = id >= p.g0 && id < p.g0 + p.El && id >= 0 && id < p.E ? id - p.g0 : -1;
    r.local[s] = e;
    if (e >= 0) atomicAdd(&r.count[e], 1);
  }
  __syncthreads();
  if (tid < 64) {                                  // wave 0: compaction
    int at = 0;
    for (int b = 0; b < p.El; b += 64) {
      const bool in = b + tid < p.El && r.count[b + tid] > 0;
      const uint64_t mask = __ballot(in);
      if (in) r.met[at + __popcll(mask & ((1ull << tid) - 1))] = b + tid;
      at += __popcll(mask);
    }
    if (tid == 0) r.n_met = at;
  }
  __syncthreads();
}

// The slots of local expert e, ascending, into list; returns their number.
// (Wave 0 scans in order, so the order does not depend on timing.)
__device__ int slots_of(const FfnArgs& p, const Routing& r, int e, int* list) {
  __syncthreads();
  const int n = p.T * p.k, tid = threadIdx.x;
  if (tid < 64) {
    int at = 0;
    for (int b = 0; b < n; b += 64) {
      const bool in = b + tid < n && r.local[b + tid] == e;
      const uint64_t mask = __ballot(in);
      if (in) list[at + __popcll(mask & ((1ull << tid) - 1))] = b + tid;
      at += __popcll(mask);
    }
  }
  __syncthreads();
  return r.count[e];
}

__device__ __forceinline__ bf8 as_bf8(uint4 v) { return __builtin_bit_cast(bf8, v); }

// Eight e4m3 codes (two words) to bfloat16, exactly.
__device__ __forceinline__ bf8 bf16_of_e4m3(uint32_t a, uint32_t b) {
  const bf2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// Eight e2m1 codes (one word) times a power of two to bfloat16, exactly.
__device__ __forceinline__ bf8 bf16_of_e2m1(uint32_t a, float s) {
  const bf2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 0);
  const bf2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 1);
  const bf2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 2);
  const bf2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 3);
  return bf8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

__device__ __forceinline__ v4f mfma_bf16(const bf8& a, const bf8& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One wave's part of R row blocks of 16 channels against up to 16 slots: the
// chunks of 128 of the contraction, `first`, first + 4, ...  A lane holds
// channel l%16; with e4m3 two 16-byte pieces a chunk, at 16 (l/16) and
// 64 + 16 (l/16); with 4 bits one piece, block l/16.  xs gives the slot's
// rows (P pieces of the same values' significance, added up).
template <bool MX4, int R, int P>
__device__ __forceinline__ void multiply(const uint8_t* const (&wrow)[R], const void* const (&wscale)[R], int nb, int cstep,
                                         int kb, int64_t K, const uint16_t* const (&xrow)[P], int first, int lane, v4f (&acc)[R]) {
  const int grp = lane >> 4;
  const int chunks = static_cast<int>((K + 127) / 128);
  const int64_t per_block = K / kb;                // e4m3: contraction elements a scale
  for (int c = first; c < chunks; c += kWaves) {
    if constexpr (MX4) {
      const int64_t k = 128 * static_cast<int64_t>(c) + 32 * grp;
      const bool in = k < K;
      bf8 xv[P][4];
#pragma unroll
      for (int q = 0; q < P; ++q)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          xv[q][u] = as_bf8(in ? *reinterpret_cast<const uint4*>(xrow[q] + k + 8 * u) : make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 w = in ? *reinterpret_cast<const uint4*>(wrow[r] + k / 2) : make_uint4(0, 0, 0, 0);
        const float s = in ? mx4::scale_value(static_cast<const uint8_t*>(wscale[r])[k / 32]) : 1.0f;
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bf8 wv = bf16_of_e2m1(ww[u], s);
#pragma unroll
          for (int q = 0; q < P; ++q) acc[r] = mfma_bf16(wv, xv[q][u], acc[r]);
        }
      }
    } else {
      bf8 xv[P][4];
      uint4 w[R][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t k = 128 * static_cast<int64_t>(c) + 64 * u + 16 * grp;
        const bool in = k < K;
#pragma unroll
        for (int q = 0; q < P; ++q)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            xv[q][2 * u + v] = as_bf8(in ? *reinterpret_cast<const uint4*>(xrow[q] + k + 8 * v) : make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int r = 0; r < R; ++r) w[r][u] = in ? *reinterpret_cast<const uint4*>(wrow[r] + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v4f part = v4f{0.f, 0.f, 0.f, 0.f};
        const uint32_t ww[8] = {w[r][0].x, w[r][0].y, w[r][0].z, w[r][0].w, w[r][1].x, w[r][1].y, w[r][1].z, w[r][1].w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bf8 wv = bf16_of_e4m3(ww[2 * u], ww[2 * u + 1]);
#pragma unroll
          for (int q = 0; q < P; ++q) part = mfma_bf16(wv, xv[q][u], part);
        }
        // several K blocks: a chunk lies in one, and its scale (a channel's own, or one for all sixteen)
        // multiplies the chunk's sum; one K block: the channel's scale comes at the end
        if (kb > 1) {
          const float* s = static_cast<const float*>(wscale[r]) + (128 * static_cast<int64_t>(c) / per_block) * nb;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(s[cstep * (4 * grp + i)], part[i], acc[r][i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][i] += part[i];
        }
      }
    }
  }
}

// Sum of the four waves' parts of a 16 x 16 block: element (channel c, slot s).
__device__ __forceinline__ float block_sum(const float (&red)[kWaves][16][17], int c, int s) {
  return (red[0][c][s] + red[1][c][s]) + (red[2][c][s] + red[3][c][s]);
}

__device__ __forceinline__ float scale_of(const void* s, int e, int kb, int nb, int64_t N, int64_t n) {
  // one K block: the channel's own factor, or its column block's
  return kb > 1 ? 1.0f : static_cast<const float*>(s)[static_cast<int64_t>(e) * nb + n / (N / nb)];
}

template <bool MX4>
__global__ __launch_bounds__(kThreads) void ffn_up_kernel(const FfnArgs p) {
  __shared__ Routing rt;
  __shared__ int list[kMaxSlots];
  __shared__ float red[2][kWaves][16][17];
  read_routing(p, rt);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l15 = lane & 15;
  const int64_t H = p.H, I = p.I, slots = static_cast<int64_t>(p.T) * p.k;
  const int tiles = static_cast<int>((I + 15) / 16);
  const int64_t rowb = MX4 ? H / 2 : H;
  for (int item = blockIdx.x; item < rt.n_met * tiles; item += gridDim.x) {
    const int e = rt.met[item / tiles];
    const int64_t c0 = 16 * static_cast<int64_t>(item % tiles);
    const int ns = slots_of(p, rt, e, list);
    const int64_t ch = min(c0 + l15, I - 1);
    const uint8_t* wrow[2];
    const void* wsc[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t n = static_cast<int64_t>(r) * I + ch;
      wrow[r] = p.w01 + (static_cast<int64_t>(e) * 2 * I + n) * rowb;
      if (MX4)
        wsc[r] = static_cast<const uint8_t*>(p.s01) + (static_cast<int64_t>(e) * 2 * I + n) * (H / 32);
      else
        wsc[r] = static_cast<const float*>(p.s01) + static_cast<int64_t>(e) * p.kb01 * p.nb01 +
                 (static_cast<int64_t>(r) * I + c0) / (2 * I / p.nb01);
    }
    for (int s0 = 0; s0 < ns; s0 += 16) {
      const int slot = list[min(s0 + l15, ns - 1)];
      const uint16_t* xrow[1] = {p.x + static_cast<int64_t>(slot / p.k) * p.ldx};
      v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
      multiply<MX4, 2, 1>(wrow, wsc, p.nb01, p.nb01 == 2 * I, MX4 ? 1 : p.kb01, H, xrow, wave, lane, acc);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[r][wave][4 * (lane >> 4) + i][l15] = acc[r][i];
      __syncthreads();
      const int c = tid & 15, s = tid >> 4;        // 256 threads: one element each
      if (s0 + s < ns && c0 + c < I) {
        float a = block_sum(red[0], c, s), b = block_sum(red[1], c, s);
        if (!MX4) {
          a *= scale_of(p.s01, e, p.kb01, p.nb01, 2 * I, c0 + c);
          b *= scale_of(p.s01, e, p.kb01, p.nb01, 2 * I, I + c0 + c);
        }
        const float hv = a / (1.0f + expf(-a)) * b;
        const uint16_t hi = f32_to_bf16(hv);
        const float rest = hv - bf16_to_f32(hi);   // not finite: the high piece alone says so
        const uint16_t lo = fabsf(rest) < INFINITY ? f32_to_bf16(rest) : 0;
        const int64_t at = static_cast<int64_t>(list[s0 + s]) * I + c0 + c;
        p.h[at] = hi;
        p.h[slots * I + at] = lo;
      }
      __syncthreads();
    }
  }
}

// y between workgroups that may sit on different XCDs: device-scope accesses.
__device__ __forceinline__ void y_store(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float y_load(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool MX4>
__global__ __launch_bounds__(kThreads) void ffn_down_kernel(const FfnArgs p) {
  __shared__ Routing rt;
  __shared__ int list[kMaxSlots];
  __shared__ float red[2][kWaves][16][17];
  __shared__ int is_last;
  read_routing(p, rt);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l15 = lane & 15;
  const int64_t H = p.H, I = p.I, slots = static_cast<int64_t>(p.T) * p.k;
  const int tiles = static_cast<int>((H + 31) / 32);
  const int64_t rowb = MX4 ? I / 2 : I;
  const int n_met = rt.n_met;
  for (int item = blockIdx.x; item < max(n_met, 1) * tiles; item += gridDim.x) {
    const int tile = item % tiles;
    const int64_t c0 = 32 * static_cast<int64_t>(tile);
    if (n_met > 0) {
      const int e = rt.met[item / tiles];
      const int ns = slots_of(p, rt, e, list);
      const uint8_t* wrow[2];
      const void* wsc[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t n = min(c0 + 16 * r + l15, H - 1);
        wrow[r] = p.wo + (static_cast<int64_t>(e) * H + n) * rowb;
        if (MX4)
          wsc[r] = static_cast<const uint8_t*>(p.so) + (static_cast<int64_t>(e) * H + n) * (I / 32);
        else
          wsc[r] = static_cast<const float*>(p.so) + static_cast<int64_t>(e) * p.kbo * p.nbo + min(c0 + 16 * r, H - 16) / (H / p.nbo);
      }
      for (int s0 = 0; s0 < ns; s0 += 16) {
        const int64_t slot = list[min(s0 + l15, ns - 1)];
        const uint16_t* xrow[2] = {p.h + slot * I, p.h + (slots + slot) * I};
        v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
        multiply<MX4, 2, 2>(wrow, wsc, p.nbo, p.nbo == H, MX4 ? 1 : p.kbo, I, xrow, wave, lane, acc);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) red[r][wave][4 * (lane >> 4) + i][l15] = acc[r][i];
        __syncthreads();
        const int c = tid & 15, s = tid >> 4;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int64_t n = c0 + 16 * r + c;
          if (s0 + s < ns && n < H) {
            float v = block_sum(red[r], c, s);
            if (!MX4) v *= scale_of(p.so, e, p.kbo, p.nbo, H, n);
            y_store(p.y + static_cast<int64_t>(list[s0 + s]) * H + n, v);
          }
        }
        __syncthreads();
      }
      __builtin_amdgcn_s_waitcnt(0);               // this wave's y has reached the coherent level
      __syncthreads();                             // ... and every wave's
      if (tid == 0) {
        is_last = atomicAdd(p.cnt + tile, 1) == n_met - 1;
        if (is_last) __hip_atomic_store(p.cnt + tile, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (!is_last) continue;
    }
    for (int i = tid; i < p.T * 32; i += kThreads) {
      const int t = i >> 5;
      const int64_t n = c0 + (i & 31);
      if (n >= H) continue;
      float v = 0.0f;
      for (int j = 0; j < p.k; ++j) {
        const int s = t * p.k + j;
        if (rt.local[s] >= 0) v = fmaf(p.tw[s], y_load(p.y + static_cast<int64_t>(s) * H + n), v);
      }
      if (p.out_bf16)
        static_cast<uint16_t*>(p.out)[t * H + n] = f32_to_bf16(v);
      else
        static_cast<float*>(p.out)[t * H + n] = v;
    }
  }
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Error word, one counter per column block, the hidden pieces, the slots' outputs.
size_t ffn_tokens_ws_bytes(int64_t slots, int64_t H, int64_t I) {
  return static_cast<size_t>(kHeader + align256(4 * moe_cdiv(H, 32)) + align256(4 * slots * I) + align256(4 * slots * H));
}

namespace {
int weight_blocks(int64_t K, int64_t N, int32_t kb, int32_t nb) {
  if (kb <= 0 || nb <= 0 || K % kb || N % nb) return MOE_ERR_SHAPE;
  if (kb > 1 && (K / kb) % 128) return MOE_ERR_UNSUPPORTED;
  if (nb != 1 && nb != N && (N / nb) % 128) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
}  // namespace
}  // namespace moe

extern "C" int moe_ffn_tokens(const void* x, int64_t ldx, const int32_t* expert_ids, const float* topk_weights, int64_t T,
                              int32_t k, int64_t H, int64_t I, int32_t E, int32_t group_offset,
                              int32_t num_local_experts, int w_format, const uint8_t* w01, const void* w01_scale,
                              int32_t kb01, int32_t nb01, const uint8_t* wo, const void* wo_scale, int32_t kbo,
                              int32_t nbo, int out_dtype, void* out, void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  if (w_format != MOE_E4M3FN && w_format != MOE_MX4) return MOE_ERR_UNSUPPORTED;
  const bool mx = w_format == MOE_MX4;
  const int64_t unit = mx ? 32 : 16;
  if (T < 0 || k <= 0 || H <= 0 || I <= 0 || H % unit || I % unit || ldx < H || ldx % 8) return MOE_ERR_SHAPE;
  if (E <= 0 || E > 1024 || group_offset < 0 || num_local_experts < 0 || group_offset + num_local_experts > E)
    return MOE_ERR_SHAPE;
  if (H > (int64_t{1} << 20) || I > (int64_t{1} << 20)) return MOE_ERR_SHAPE;   // item counts stay below 2^31
  if (mx) {
    if (kb01 || nb01 || kbo || nbo) return MOE_ERR_UNSUPPORTED;
  } else {
    const int c0 = weight_blocks(H, 2 * I, kb01, nb01), c1 = weight_blocks(I, H, kbo, nbo);
    if (c0 != MOE_OK) return c0;
    if (c1 != MOE_OK) return c1;
  }
  if (out_dtype == MOE_DTYPE_DEFAULT || out_dtype == MOE_E4M3FN) out_dtype = MOE_BF16;
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (T > kMaxT || T * k > kMaxSlots) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !expert_ids || !topk_weights || !out) return MOE_ERR_NULL;
  if (num_local_experts > 0 && (!w01 || !w01_scale || !wo || !wo_scale)) return MOE_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(w01) % 16 || reinterpret_cast<uintptr_t>(wo) % 16)
    return MOE_ERR_SHAPE;
  const int64_t slots = T * k;
  if (!ws || ws_bytes < ffn_tokens_ws_bytes(slots, H, I)) return MOE_ERR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  const int64_t cnt_off = kHeader, h_off = cnt_off + align256(4 * moe_cdiv(H, 32)), y_off = h_off + align256(4 * slots * I);
  const FfnArgs p{static_cast<const uint16_t*>(x), ldx, expert_ids, topk_weights, static_cast<int>(T), k, H, I, E,
                  group_offset, num_local_experts, w01, w01_scale, kb01, nb01, wo, wo_scale, kbo, nbo, out,
                  out_dtype == MOE_BF16, reinterpret_cast<int32_t*>(base), reinterpret_cast<int32_t*>(base + cnt_off),
                  reinterpret_cast<uint16_t*>(base + h_off), reinterpret_cast<float*>(base + y_off)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t most = slots < num_local_experts ? slots : num_local_experts;      // experts that can be met
  const int64_t cap = 8 * tile::num_cus();
  const int64_t up = most * moe_cdiv(I, 16), down = (most > 0 ? most : 1) * moe_cdiv(H, 32);
  const unsigned gu = static_cast<unsigned>(up < 1 ? 1 : up < cap ? up : cap), gd = static_cast<unsigned>(down < cap ? down : cap);
  if (mx) {
    ffn_up_kernel<true><<<gu, kThreads, 0, st>>>(p);
    MOE_CHECK_LAUNCH();
    ffn_down_kernel<true><<<gd, kThreads, 0, st>>>(p);
  } else {
    ffn_up_kernel<false><<<gu, kThreads, 0, st>>>(p);
    MOE_CHECK_LAUNCH();
    ffn_down_kernel<false><<<gd, kThreads, 0, st>>>(p);
  }
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
