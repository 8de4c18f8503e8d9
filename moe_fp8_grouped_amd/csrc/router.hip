// moe_router_topk / moe_router_topk_backward: the router in front of the
// sort, from a token's logits z [E] to its k experts and their weights, and
// the gradient back to the logits.
//   scores   softmax p_e = exp(z_e - m) / sum_f exp(z_f - m), m = max z, or
//            sigmoid p_e = 1 / (1 + exp(-z_e))
//   choice   the k largest z_e (scores rise with the logits, so no rounding
//            of a score decides), or with a bias the k largest p_e + b_e,
//            formed in 64 bits; equal keys go to the lower expert
//   weights  scale * p_e, or scale * p_e / (sum of the chosen p)
// A logit of -inf (or NaN) takes its expert out: it is chosen after every
// other one and its weight is 0.
#include "common.hpp"

namespace moe {
namespace {

constexpr int kMaxE = 1024, kMaxK = 64;

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* z, int64_t i) {
  return BF16 ? bf16_to_f32(static_cast<const uint16_t*>(z)[i]) : static_cast<const float*>(z)[i];
}

// -inf and NaN both take an expert out.
__device__ __forceinline__ float masked(float z) { return z != z ? -INFINITY : z; }

// Monotone unsigned keys: a larger key is a larger value; 0 is below all.
__device__ __forceinline__ uint64_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);             // -0 and +0 are equal keys
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// One wave per row, expert e = lane + 64 i in register i.
template <bool BF16, int V, bool BIAS, bool SIGMOID>
__global__ __launch_bounds__(256) void router_topk_kernel(const void* __restrict__ logits, int64_t ldl, int64_t T, int E,
                                                          int k, const float* __restrict__ bias, int renorm, float scale,
                                                          int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  float z[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    z[i] = e < E ? masked(load_logit<BF16>(logits, t * ldl + e)) : -INFINITY;
  }
  float m = z[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, z[i]);
  m = wave_max(m);
  const float m0 = m == -INFINITY ? 0.0f : m;
  // softmax's denominator (64-bit where a bias is added to the scores)
  float sum = 0.0f;
  double dsum = 0.0;
  double p[V];
  if constexpr (!SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (BIAS) {
        p[i] = exp(static_cast<double>(z[i]) - static_cast<double>(m0));
        dsum += p[i];
      }
      sum += expf(z[i] - m0);
    }
    sum = wave_sum(sum);
    if constexpr (BIAS) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) dsum += __shfl_xor(dsum, o, MOE_WAVE);
    }
  }
  uint64_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    if constexpr (BIAS) {
      const double s = SIGMOID ? 1.0 / (1.0 + exp(-static_cast<double>(z[i]))) : p[i] / dsum;
      const bool in = z[i] > -INFINITY;
      key[i] = e >= E ? 0 : order_key(in ? s + static_cast<double>(bias[e < E ? e : 0]) : -static_cast<double>(INFINITY));
    } else {
      key[i] = e >= E ? 0 : order_key(z[i]);
    }
  }
  float my_z = -INFINITY;                    // lane j: the j-th choice
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t bk = 0;
    int bi = kMaxE;
    float bz = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (key[i] > bk) { bk = key[i]; bi = lane + 64 * i; bz = z[i]; }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t ok = __shfl_xor(bk, o, MOE_WAVE);
      const int oi = __shfl_xor(bi, o, MOE_WAVE);
      const float oz = __shfl_xor(bz, o, MOE_WAVE);
      if (ok > bk || (ok == bk && oi < bi)) { bk = ok; bi = oi; bz = oz; }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (bi == lane + 64 * i) key[i] = 0;
    if (lane == j) { my_z = bz; my_id = bi; }
  }
  float w;
  if (SIGMOID) {
    w = 1.0f / (1.0f + expf(-my_z));
  } else {
    const float top = wave_max(my_z);        // renormalised softmax: a softmax over the chosen
    const float base = renorm ? (top == -INFINITY ? 0.0f : top) : m0;
    w = expf(my_z - base);
    if (!renorm) w = sum > 0.0f ? w / sum : 0.0f;
  }
  if (lane >= k) w = 0.0f;
  if (renorm) {
    const float tot = wave_sum(w);
    w = tot > 0.0f ? w / tot : 0.0f;
  }
  if (lane < k) {
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = scale * w;
  }
}

// The gradient, the choice held fixed: with g_j = scale * dw_j,
//   softmax           dz_e = p_e (g_e - sum_j g_j p_j), g_e = 0 unless chosen
//   softmax, renorm.  dz_e = r_e (g_e - sum_j g_j r_j) for the chosen, r = their softmax
//   sigmoid           dz_e = g_e p_e (1 - p_e)
//   sigmoid, renorm.  the same with (g_e - sum_j g_j p_j / S) / S for g_e, S = sum of the chosen p
// An index outside [0, E) takes no part; an index given twice counts twice.
template <bool BF16, int V, bool SIGMOID>
__global__ __launch_bounds__(256) void router_bwd_kernel(const void* __restrict__ logits, int64_t ldl,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ dweights, int64_t T, int E, int k,
                                                         int renorm, float scale, void* __restrict__ dlogits,
                                                         int64_t ldd) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  float z[V], g[V], n[V];                    // n: how often the expert was chosen
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    z[i] = e < E ? masked(load_logit<BF16>(logits, t * ldl + e)) : -INFINITY;
    g[i] = 0.0f;
    n[i] = 0.0f;
  }
  const int id_l = lane < k ? ids[t * k + lane] : -1;
  const float dw_l = lane < k ? dweights[t * k + lane] * scale : 0.0f;
  for (int j = 0; j < k; ++j) {
    const int id = __shfl(id_l, j, MOE_WAVE);
    const float dw = __shfl(dw_l, j, MOE_WAVE);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (id == lane + 64 * i && id < E) { g[i] += dw; n[i] += 1.0f; }
  }
  float m = -INFINITY;                       // over all experts, or the chosen ones
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, (!renorm || n[i] > 0.0f) ? z[i] : -INFINITY);
  m = wave_max(m);
  const float m0 = m == -INFINITY ? 0.0f : m;
  float p[V], sum = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (SIGMOID) {
      p[i] = 1.0f / (1.0f + expf(-z[i]));
      sum += n[i] * p[i];
    } else {
      p[i] = renorm && n[i] == 0.0f ? 0.0f : expf(z[i] - m0);
      sum += renorm ? n[i] * p[i] : p[i];
    }
    dot += g[i] * p[i];
  }
  sum = wave_sum(sum);
  dot = wave_sum(dot);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    if (e >= E) continue;
    float d;
    if (SIGMOID) {
      const float ge = renorm ? (g[i] - n[i] * (dot * inv)) * inv : g[i];
      d = ge * p[i] * (1.0f / (1.0f + expf(z[i])));        // 1 - p without cancellation
    } else {
      d = p[i] * inv * (g[i] - (renorm ? n[i] : 1.0f) * (dot * inv));
    }
    if (BF16)
      static_cast<uint16_t*>(dlogits)[t * ldd + e] = f32_to_bf16(d);
    else
      static_cast<float*>(dlogits)[t * ldd + e] = d;
  }
}

template <bool BF16, int V>
hipError_t launch_topk(const void* z, int64_t ldl, int64_t T, int E, int k, int score, const float* bias, int renorm,
                       float scale, int32_t* ids, float* w, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(moe_cdiv(T, 4));
  const bool sig = score == MOE_SCORE_SIGMOID;
#define MOE_ROUTER(B, S) router_topk_kernel<BF16, V, B, S><<<grid, 256, 0, st>>>(z, ldl, T, E, k, bias, renorm, scale, ids, w)
  if (bias) { if (sig) MOE_ROUTER(true, true); else MOE_ROUTER(true, false); }
  else { if (sig) MOE_ROUTER(false, true); else MOE_ROUTER(false, false); }
#undef MOE_ROUTER
  return hipGetLastError();
}

template <bool BF16, int V>
hipError_t launch_bwd(const void* z, int64_t ldl, const int32_t* ids, const float* dw, int64_t T, int E, int k,
                      int score, int renorm, float scale, void* dz, int64_t ldd, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(moe_cdiv(T, 4));
  if (score == MOE_SCORE_SIGMOID)
    router_bwd_kernel<BF16, V, true><<<grid, 256, 0, st>>>(z, ldl, ids, dw, T, E, k, renorm, scale, dz, ldd);
  else
    router_bwd_kernel<BF16, V, false><<<grid, 256, 0, st>>>(z, ldl, ids, dw, T, E, k, renorm, scale, dz, ldd);
  return hipGetLastError();
}

int router_check(int dtype, int64_t ldl, int64_t T, int32_t E, int32_t k, int score, int renorm, float scale) {
  if (T < 0 || E <= 0 || E > kMaxE || k <= 0 || k > kMaxK || k > E || ldl < E) return MOE_ERR_SHAPE;
  if (T > (int64_t{1} << 31)) return MOE_ERR_SHAPE;         // a wave a row: the grid stays below 2^31 workgroups
  if (!(scale > 0.0f) || !(scale <= 3.402823466e38f)) return MOE_ERR_SHAPE;
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (renorm != 0 && renorm != 1) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

#define MOE_BY_V(CALL)                       \
  (E <= 64 ? CALL(1) : E <= 128 ? CALL(2) : E <= 256 ? CALL(4) : E <= 512 ? CALL(8) : CALL(16))

extern "C" int moe_router_topk(const void* logits, int logits_dtype, int64_t ldl, int64_t T, int32_t E, int32_t k,
                               int score, const float* select_bias, int renormalize, float weight_scale,
                               int32_t* expert_ids, float* topk_weights, void* stream) {
  const int c = moe::router_check(logits_dtype, ldl, T, E, k, score, renormalize, weight_scale);
  if (c != MOE_OK) return c;
  if (T == 0) return MOE_OK;
  if (!logits || !expert_ids || !topk_weights) return MOE_ERR_NULL;
  hipStream_t st = static_cast<hipStream_t>(stream);
#define MOE_B(V) moe::launch_topk<true, V>(logits, ldl, T, E, k, score, select_bias, renormalize, weight_scale, expert_ids, topk_weights, st)
#define MOE_F(V) moe::launch_topk<false, V>(logits, ldl, T, E, k, score, select_bias, renormalize, weight_scale, expert_ids, topk_weights, st)
  const hipError_t e = logits_dtype == MOE_BF16 ? MOE_BY_V(MOE_B) : MOE_BY_V(MOE_F);
#undef MOE_B
#undef MOE_F
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

extern "C" int moe_router_topk_backward(const void* logits, int logits_dtype, int64_t ldl, const int32_t* expert_ids,
                                        const float* dweights, int64_t T, int32_t E, int32_t k, int score,
                                        int renormalize, float weight_scale, void* dlogits, int64_t ldd, void* stream) {
  const int c = moe::router_check(logits_dtype, ldl, T, E, k, score, renormalize, weight_scale);
  if (c != MOE_OK) return c;
  if (ldd < E) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!logits || !expert_ids || !dweights || !dlogits) return MOE_ERR_NULL;
  hipStream_t st = static_cast<hipStream_t>(stream);
#define MOE_B(V) moe::launch_bwd<true, V>(logits, ldl, expert_ids, dweights, T, E, k, score, renormalize, weight_scale, dlogits, ldd, st)
#define MOE_F(V) moe::launch_bwd<false, V>(logits, ldl, expert_ids, dweights, T, E, k, score, renormalize, weight_scale, dlogits, ldd, st)
  const hipError_t e = logits_dtype == MOE_BF16 ? MOE_BY_V(MOE_B) : MOE_BY_V(MOE_F);
#undef MOE_B
#undef MOE_F
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
