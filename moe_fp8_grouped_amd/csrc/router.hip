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
#include "wave_common.hpp"

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
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);             // -0 and +0 are equal keys
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// Sigmoids of renormalised weights where a chosen logit is below kLow: there
// exp(-z) passes float32's range and p falls below its normal one, while the
// ratios of the chosen p are ordinary numbers.  So p times one factor for the
// row: with top, the largest chosen logit, below kLow too, p = exp(z) to
// 2^-92 and the factor is exp(-top); otherwise it is 2^100.  The differences
// z - top and z - kLow are exact wherever the result is not 0.  Below kNone p
// is 0: a mask of the type's lowest value is no logit to compare with another.
constexpr float kLow = -64.0f, kNone = -700.0f;
__device__ __forceinline__ bool is_low(float z) { return z < kLow && z >= kNone; }
__device__ __forceinline__ float sigmoid_times(float z, float top) {
  if (z < kNone) return 0.0f;
  if (top < kLow) return expf(z - top);
  constexpr float kBig = 1267650600228229401496703205376.0f;          // 2^100
  constexpr float kBigLow = 203.30718f;                               // 2^100 exp(kLow)
  return z < kLow ? expf(z - kLow) * kBigLow : kBig / (1.0f + expf(-z));
}

// sigmoid(z), and 1 - sigmoid(z) without cancellation, from exp(-|z|), which stays in range
__device__ __forceinline__ float sigmoid(float z, float& rest) {
  const float e = expf(-fabsf(z)), near = 1.0f / (1.0f + e), far = e / (1.0f + e);
  rest = z < 0.0f ? near : far;
  return z < 0.0f ? far : near;
}

// One wave per row, expert e = lane + 64 i in register i.  Every choice is one
// maximum over the wave (two for the bias's 64-bit keys), and ballots that find
// its first expert.  8192 rows of 256 bf16 logits, k = 8: 8.5 us in the
// trace (as a graph of one call 10.2, where choices through LDS shuffles of key,
// expert and logit took 25); what is left is instructions, not the 0.9 us of
// bytes.
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
  m = max_of(m);
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
    sum = sum_of(sum);
    if constexpr (BIAS) dsum = sum_of(dsum);
  }
  // keys by halves; without a bias the upper one says all
  uint32_t hi[V], lo[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    uint64_t key;
    if constexpr (BIAS) {
      const double s = SIGMOID ? 1.0 / (1.0 + exp(-static_cast<double>(z[i]))) : p[i] / dsum;
      const bool in = z[i] > -INFINITY;
      key = order_key(in ? s + static_cast<double>(bias[e < E ? e : 0]) : -static_cast<double>(INFINITY));
    } else {
      key = static_cast<uint64_t>(order_key(z[i])) << 32;
    }
    hi[i] = e < E ? max(static_cast<uint32_t>(key >> 32), 1u) : 0;   // (0: no expert, or chosen; a NaN's key may be 0 too)
    lo[i] = static_cast<uint32_t>(key);
  }
  float my_z = -INFINITY;                    // lane j: the j-th choice
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t top = hi[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max(top, hi[i]);
    top = max_of(top);
    uint32_t low = 0;
    if constexpr (BIAS) {
#pragma unroll
      for (int i = 0; i < V; ++i) low = max(low, hi[i] == top ? lo[i] : 0u);
      low = max_of(low);
    }
    bool found = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {            // experts in order
      const uint64_t at = __ballot(hi[i] == top && (!BIAS || lo[i] == low));
      if (!found && at) {
        found = true;
        const int l = __builtin_ctzll(at);
        if (lane == j) my_id = l + 64 * i;
        const float zl = from_lane(z[i], l);
        if (lane == j) my_z = zl;
        if (lane == l) hi[i] = 0;
      }
    }
  }
  float w;
  if (SIGMOID) {
    float rest;
    w = sigmoid(my_z, rest);
    if (renorm && __any(is_low(my_z))) w = sigmoid_times(my_z, max_of(my_z));
  } else {
    const float top = max_of(my_z);        // renormalised softmax: a softmax over the chosen
    const float base = renorm ? (top == -INFINITY ? 0.0f : top) : m0;
    w = expf(my_z - base);
    if (!renorm) w = sum > 0.0f ? w / sum : 0.0f;
  }
  if (lane >= k) w = 0.0f;
  if (renorm) {
    const float tot = sum_of(w);
    w = tot > 0.0f ? w / tot : 0.0f;
  }
  if (lane < k) {
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = scale * w;
  }
}

// The gradient, one wave a row, the choice held fixed: with g_j = scale * dw_j,
//   softmax           dz_e = p_e (g_e - sum_j g_j p_j), g_e = 0 unless chosen
//   softmax, renorm.  dz_e = r_e (g_e - sum_j g_j r_j) for the chosen, r = their softmax
//   sigmoid           dz_e = g_e p_e (1 - p_e)
//   sigmoid, renorm.  the same with (g_e - sum_j g_j p_j / S) / S for g_e, S = sum of the chosen p
// An index outside [0, E) takes no part; an index given twice counts twice.
// An expert that was taken out has gradient 0 and its slots' gradients take
// no part: a padded token's may hold anything.
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
    const int id = __builtin_amdgcn_readlane(id_l, j);
    const float dw = from_lane(dw_l, j);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (id == lane + 64 * i && id < E) { g[i] += dw; n[i] += 1.0f; }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) g[i] = z[i] == -INFINITY ? 0.0f : g[i];        // taken out: a gradient of any value counts nothing
  float m = -INFINITY;                       // over all experts, or the chosen ones
  bool low = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    m = fmaxf(m, (!renorm || n[i] > 0.0f) ? z[i] : -INFINITY);
    low |= n[i] > 0.0f && is_low(z[i]);
  }
  m = max_of(m);
  low = SIGMOID && renorm && __any(low);
  const float m0 = m == -INFINITY ? 0.0f : m;
  float p[V], rest[SIGMOID ? V : 1], sum = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (SIGMOID) {
      p[i] = sigmoid(z[i], rest[i]);
      if (low) p[i] = n[i] > 0.0f ? sigmoid_times(z[i], m) : 0.0f;
      sum += n[i] * p[i];
    } else {
      p[i] = renorm && n[i] == 0.0f ? 0.0f : expf(z[i] - m0);
      sum += renorm ? n[i] * p[i] : p[i];
    }
    if (!low) dot += g[i] * p[i];
  }
  sum = sum_of(sum);
  if (low) {                                 // the ratios first: times the factor a gradient could leave the range
    const float inv_sum = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] *= inv_sum;
      dot += g[i] * p[i];
    }
    sum = 1.0f;
  }
  dot = sum_of(dot);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    if (e >= E) continue;
    float d;
    if constexpr (SIGMOID) {
      d = (renorm ? (g[i] - n[i] * (dot * inv)) * (p[i] * inv) : g[i] * p[i]) * rest[i];
    } else {
      d = p[i] * inv * (g[i] - (renorm ? n[i] : 1.0f) * (dot * inv));
    }
    if (z[i] == -INFINITY) d = 0.0f;
    if (BF16)
      static_cast<uint16_t*>(dlogits)[t * ldd + e] = f32_to_bf16(d);
    else
      static_cast<float*>(dlogits)[t * ldd + e] = d;
  }
}

// The same for up to 128 experts: sixteen lanes a row, four neighbouring
// experts a lane and V times that, four rows a wave.  One wave a row spends its
// instructions on idle lanes and on reductions over rows that hold little:
// 32768 rows of 64 float32 logits, k = 8, 14.0 us against 9.6 as graphs of one
// call (8.4 in the trace; the bytes alone 3.6; what is left is the launch and
// instructions).
template <bool BF16, int V, bool SIGMOID>
__global__ __launch_bounds__(256) void router_bwd_rows_kernel(const void* __restrict__ logits, int64_t ldl,
                                                              const int32_t* __restrict__ ids,
                                                              const float* __restrict__ dweights, int64_t T, int E, int k,
                                                              int renorm, float scale, void* __restrict__ dlogits,
                                                              int64_t ldd, bool wide) {
  const int lane = threadIdx.x & 63, sub = lane & 15;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6)) * 4 + (lane >> 4);
  const int64_t t = min(row, T - 1);         // (past the last row: its copy, not stored)
  float z[V][4], g[V][4], n[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 64 * i + 4 * sub;
    if (wide && e < E) {                     // whole, aligned vectors of four
      if (BF16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + t * ldl + e);
        z[i][0] = masked(__uint_as_float(v.x << 16));
        z[i][1] = masked(__uint_as_float(v.x & 0xffff0000u));
        z[i][2] = masked(__uint_as_float(v.y << 16));
        z[i][3] = masked(__uint_as_float(v.y & 0xffff0000u));
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + t * ldl + e);
        z[i][0] = masked(v.x);
        z[i][1] = masked(v.y);
        z[i][2] = masked(v.z);
        z[i][3] = masked(v.w);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) z[i][c] = e + c < E ? masked(load_logit<BF16>(logits, t * ldl + e + c)) : -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) g[i][c] = n[i][c] = 0.0f;
  }
  for (int j0 = 0; j0 < k; j0 += 16) {
    int id_l = j0 + sub < k ? ids[t * k + j0 + sub] : -1;
    const float dw_l = j0 + sub < k ? dweights[t * k + j0 + sub] * scale : 0.0f;
    if (id_l >= E) id_l = -1;
    const int stop = min(16, k - j0);
    for (int j = 0; j < stop; ++j) {
      const int d = __shfl(id_l, (lane & 48) + j, MOE_WAVE) - 4 * sub;
      const float dw = __shfl(dw_l, (lane & 48) + j, MOE_WAVE);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (d == 64 * i + c) { g[i][c] += dw; n[i][c] += 1.0f; }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) g[i][c] = z[i][c] == -INFINITY ? 0.0f : g[i][c];   // taken out: a gradient of any value counts nothing
  float m0 = -INFINITY;
  bool low = false;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) low |= n[i][c] > 0.0f && is_low(z[i][c]);
  low = SIGMOID && renorm && row_max(low ? 1.0f : 0.0f) > 0.0f;
  if (!SIGMOID || low) {                     // the maximum over all experts, or the chosen ones
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) m0 = fmaxf(m0, (!renorm || n[i][c] > 0.0f) ? z[i][c] : -INFINITY);
    m0 = row_max(m0);
    if (m0 == -INFINITY) m0 = 0.0f;
  }
  float p[V][4], rest[SIGMOID ? V : 1][4], sum = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (SIGMOID) {
        p[i][c] = sigmoid(z[i][c], rest[i][c]);
        if (low) p[i][c] = n[i][c] > 0.0f ? sigmoid_times(z[i][c], m0) : 0.0f;
        sum += n[i][c] * p[i][c];
      } else {
        p[i][c] = renorm && n[i][c] == 0.0f ? 0.0f : expf(z[i][c] - m0);
        sum += renorm ? n[i][c] * p[i][c] : p[i][c];
      }
      if (!low) dot += g[i][c] * p[i][c];
    }
  sum = row_sum(sum);
  if (low) {                                 // the ratios first: times the factor a gradient could leave the range
    const float inv_sum = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        p[i][c] *= inv_sum;
        dot += g[i][c] * p[i][c];
      }
    sum = 1.0f;
  }
  dot = row_sum(dot);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  if (row >= T) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 64 * i + 4 * sub;
    if (e >= E) continue;
    float d[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (SIGMOID) {
        d[c] = (renorm ? (g[i][c] - n[i][c] * (dot * inv)) * (p[i][c] * inv) : g[i][c] * p[i][c]) * rest[i][c];
      } else {
        d[c] = p[i][c] * inv * (g[i][c] - (renorm ? n[i][c] : 1.0f) * (dot * inv));
      }
      if (z[i][c] == -INFINITY) d[c] = 0.0f;
    }
    if (wide) {
      if (BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dlogits) + t * ldd + e) =
            make_uint2(f32_to_bf16(d[0]) | static_cast<uint32_t>(f32_to_bf16(d[1])) << 16,
                       f32_to_bf16(d[2]) | static_cast<uint32_t>(f32_to_bf16(d[3])) << 16);
      else
        *reinterpret_cast<float4*>(static_cast<float*>(dlogits) + t * ldd + e) = make_float4(d[0], d[1], d[2], d[3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (e + c >= E) continue;
        if (BF16)
          static_cast<uint16_t*>(dlogits)[t * ldd + e + c] = f32_to_bf16(d[c]);
        else
          static_cast<float*>(dlogits)[t * ldd + e + c] = d[c];
      }
    }
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
  if constexpr (V <= 2) {
    const uintptr_t size = BF16 ? 2 : 4;
    const uintptr_t a = reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(dz) | static_cast<uintptr_t>(ldl | ldd | E) * size;
    const bool wide = a % (4 * size) == 0;
    const unsigned grid = static_cast<unsigned>(moe_cdiv(T, 16));
    if (score == MOE_SCORE_SIGMOID)
      router_bwd_rows_kernel<BF16, V, true><<<grid, 256, 0, st>>>(z, ldl, ids, dw, T, E, k, renorm, scale, dz, ldd, wide);
    else
      router_bwd_rows_kernel<BF16, V, false><<<grid, 256, 0, st>>>(z, ldl, ids, dw, T, E, k, renorm, scale, dz, ldd, wide);
  } else {
    const unsigned grid = static_cast<unsigned>(moe_cdiv(T, 4));
    if (score == MOE_SCORE_SIGMOID)
      router_bwd_kernel<BF16, V, true><<<grid, 256, 0, st>>>(z, ldl, ids, dw, T, E, k, renorm, scale, dz, ldd);
    else
      router_bwd_kernel<BF16, V, false><<<grid, 256, 0, st>>>(z, ldl, ids, dw, T, E, k, renorm, scale, dz, ldd);
  }
  return hipGetLastError();
}

int router_check(int dtype, int64_t ldl, int64_t T, int32_t E, int32_t k, int score, int renorm, float scale) {
  if (T < 0 || E <= 0 || E > kMaxE || k <= 0 || k > kMaxK || k > E || ldl < E) return MOE_ERR_SHAPE;
  if (T > (int64_t{1} << 31)) return MOE_ERR_SHAPE;
  if (!(scale > 0.0f) || !(scale <= 3.402823466e38f)) return MOE_ERR_SHAPE;
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (renorm != 0 && renorm != 1) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

// A launch takes fewer than 2^32 threads in a dimension (beyond that it runs a part of them without an error): rows by
// parts that stay below with a wave a row.
constexpr int64_t kRowsALaunch = int64_t{1} << 25;

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
  for (int64_t t = 0; t < T; t += kRowsALaunch) {
    const int64_t n = T - t < kRowsALaunch ? T - t : kRowsALaunch;
    const void* z = static_cast<const char*>(logits) + t * ldl * (logits_dtype == MOE_BF16 ? 2 : 4);
    int32_t* ids = expert_ids + t * k;
    float* w = topk_weights + t * k;
#define MOE_B(V) moe::launch_topk<true, V>(z, ldl, n, E, k, score, select_bias, renormalize, weight_scale, ids, w, st)
#define MOE_F(V) moe::launch_topk<false, V>(z, ldl, n, E, k, score, select_bias, renormalize, weight_scale, ids, w, st)
    const hipError_t e = logits_dtype == MOE_BF16 ? MOE_BY_V(MOE_B) : MOE_BY_V(MOE_F);
#undef MOE_B
#undef MOE_F
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  return MOE_OK;
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
  for (int64_t t = 0; t < T; t += kRowsALaunch) {
    const int64_t n = T - t < kRowsALaunch ? T - t : kRowsALaunch, size = logits_dtype == MOE_BF16 ? 2 : 4;
    const void* z = static_cast<const char*>(logits) + t * ldl * size;
    void* dz = static_cast<char*>(dlogits) + t * ldd * size;
    const int32_t* ids = expert_ids + t * k;
    const float* dw = dweights + t * k;
#define MOE_B(V) moe::launch_bwd<true, V>(z, ldl, ids, dw, n, E, k, score, renormalize, weight_scale, dz, ldd, st)
#define MOE_F(V) moe::launch_bwd<false, V>(z, ldl, ids, dw, n, E, k, score, renormalize, weight_scale, dz, ldd, st)
    const hipError_t e = logits_dtype == MOE_BF16 ? MOE_BY_V(MOE_B) : MOE_BY_V(MOE_F);
#undef MOE_B
#undef MOE_F
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  return MOE_OK;
}
