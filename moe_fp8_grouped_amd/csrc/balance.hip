// moe_balance_loss / moe_balance_loss_backward: how evenly a router spreads
// its tokens, per sequence, and the gradient to the logits.  With the shares
// p_t of a token's scores over the experts in service, n tokens that have one,
// and c[e] choices of expert e in the sequence:
//   loss = E / (k n^2) sum_e c[e] sum_t p[t, e]
//   dz[t, e] = dloss E / (k n^2) p_e (c[e] - sum_f c[f] p_f) r_e
// r = 1 for softmax shares, 1 - sigmoid(z) for normalised sigmoids.
#include "common.hpp"

namespace moe {
namespace {

constexpr int kMaxE = 1024, kMaxK = 64;
constexpr float kOut = -1e30f;               // a logit at or below it, or NaN, takes its expert out
constexpr int64_t kHeader = 256;             // workspace: error word

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* z, int64_t i) {
  const float v = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(z)[i]) : static_cast<const float*>(z)[i];
  return v > kOut ? v : -INFINITY;
}

// A score up to a factor common to the row, with m its largest logit: exp(z - m), or
// sigmoid(z) / exp(min(m, 0)) = exp(min(z, 0) - min(m, 0)) / (1 + exp(-|z|)),
// which stays in range where every sigmoid of the row is below it.
template <bool SIGMOID>
__device__ __forceinline__ float score(float z, float m, float& rest) {
  if constexpr (SIGMOID) {
    const float e = expf(-fabsf(z)), d = 1.0f / (1.0f + e);
    rest = z < 0.0f ? d : e * d;
    return (z < 0.0f ? expf(z - fminf(m, 0.0f)) : 1.0f) * d;
  } else {
    rest = 1.0f;
    return expf(z - m);
  }
}

__device__ __forceinline__ int clamp_offset(const int32_t* off, int64_t s, int64_t T) {
  return static_cast<int>(min(static_cast<int64_t>(max(off[s], 0)), T));
}

// The last sequence that starts at or before token t, or -1.
__device__ __forceinline__ int64_t find_sequence(const int32_t* off, int64_t S, int64_t T, int64_t t) {
  int64_t lo = -1, hi = S - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (clamp_offset(off, mid, T) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tokens of one workgroup of the forward pass.
__host__ __device__ inline int64_t chunk_tokens(int64_t T) {
  const int64_t c = (T + 1023) / 1024;
  return c < 32 ? 32 : c;
}

struct BalanceArgs {
  const void* z;
  int64_t ldl;
  const int32_t* ids;
  int64_t T;
  int E, k;
  const int32_t* off;
  int64_t S;
  float* part;                               // [chunks + S][E] share sums, then the same of counts, then of tokens
  int32_t* err;
};

// A workgroup takes a run of tokens, a wave a token at a time, and leaves the sums of
// each sequence that it meets in a slot of its own: chunk + sequence.  (From
// one piece to the next the chunk or the sequence grows, so no two pieces share a slot, and a
// sequence's slots are a run.)
template <bool BF16, bool SIGMOID, int V>
__global__ __launch_bounds__(256) void balance_kernel(const BalanceArgs p, int64_t chunk) {
  __shared__ float sums[4][64 * V];
  __shared__ int counts[64 * V], tokens;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.E;
  const int64_t slots = gridDim.x + p.S;
  float* part = p.part;
  int32_t* cpart = reinterpret_cast<int32_t*>(part + slots * E);
  int32_t* npart = cpart + slots * E;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk, t1 = min(t0 + chunk, p.T);
  int64_t s = p.off ? find_sequence(p.off, p.S, p.T, t0) : 0;
  int64_t t = t0;
  if (s < 0) {
    s = 0;
    t = max(t0, static_cast<int64_t>(clamp_offset(p.off, 0, p.T)));
  }
  for (; s < p.S && t < t1; ++s) {
    const int64_t end = p.off ? min(static_cast<int64_t>(clamp_offset(p.off, s + 1, p.T)), t1) : t1;
    if (end <= t) continue;
    for (int i = tid; i < 64 * V; i += 256) counts[i] = 0;
    if (tid == 0) tokens = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int64_t r = t + wave; r < end; r += 4) {
      float z[V], m = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        z[i] = e < E ? load_logit<BF16>(p.z, r * p.ldl + e) : -INFINITY;
        m = fmaxf(m, z[i]);
      }
      m = wave_max(m);
      if (m == -INFINITY) continue;          // a padded token
      float q[V], sum = 0.0f, rest;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        q[i] = z[i] == -INFINITY ? 0.0f : score<SIGMOID>(z[i], m, rest);
        sum += q[i];
      }
      const float inv = 1.0f / wave_sum(sum);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += q[i] * inv;
      if (lane < p.k) {
        const int id = p.ids[r * p.k + lane];
        if (id >= 0 && id < E && load_logit<BF16>(p.z, r * p.ldl + id) != -INFINITY) atomicAdd(&counts[id], 1);
      }
      if (lane == 0) atomicAdd(&tokens, 1);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][lane + 64 * i] = acc[i];
    __syncthreads();
    const int64_t slot = blockIdx.x + s;
    for (int e = tid; e < E; e += 256) {
      part[slot * E + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
      cpart[slot * E + e] = counts[e];
    }
    if (tid == 0) npart[slot] = tokens;
    __syncthreads();
    t = end;
  }
}

// A workgroup a sequence: its slots' sums in order, and the loss.
__global__ __launch_bounds__(256) void balance_join_kernel(const BalanceArgs p, int64_t chunk, int64_t chunks, float* __restrict__ loss,
                                                           int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
  __shared__ float red[4];
  const int tid = threadIdx.x, E = p.E;
  const int64_t slots = chunks + p.S;
  const float* part = p.part;
  const int32_t* cpart = reinterpret_cast<const int32_t*>(part + slots * E);
  const int32_t* npart = cpart + slots * E;
  for (int64_t s = blockIdx.x; s < p.S; s += gridDim.x) {
    int64_t b = 0, e = p.T;
    if (p.off) {
      const int32_t lo = p.off[s], hi = p.off[s + 1];
      if (tid == 0 && (lo < 0 || hi < lo || hi > p.T)) raise_error(p.err, MOE_DEVERR_SEQUENCE);
      b = clamp_offset(p.off, s, p.T);
      e = clamp_offset(p.off, s + 1, p.T);
    }
    const int64_t first = b / chunk + s, last = e > b ? (e - 1) / chunk + s : first - 1;
    int64_t n = 0;
    for (int64_t i = first; i <= last; ++i) n += npart[i];
    float dot = 0.0f;
    for (int x = tid; x < E; x += 256) {
      float sum = 0.0f;
      int64_t c = 0;
      for (int64_t i = first; i <= last; ++i) {
        sum += part[i * E + x];
        c += cpart[i * E + x];
      }
      counts[s * E + x] = static_cast<int32_t>(c);
      dot += static_cast<float>(c) * sum;
    }
    dot = wave_sum(dot);
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = dot;
    __syncthreads();
    if (tid == 0) {
      tokens[s] = static_cast<int32_t>(n);
      const double d = static_cast<double>(n);
      loss[s] = n > 0 ? static_cast<float>(static_cast<double>((red[0] + red[1]) + (red[2] + red[3])) * E / (p.k * d * d)) : 0.0f;
    }
  }
}

// One wave a token.  The counts enter less their mean, which the gradient does
// not see (the shares sum to 1) and the differences keep their digits by.
template <bool BF16, bool SIGMOID, int V>
__global__ __launch_bounds__(256) void balance_bwd_kernel(const BalanceArgs p, const int32_t* __restrict__ counts,
                                                          const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                                                          int accumulate, void* __restrict__ dz, int64_t ldd) {
  const int lane = threadIdx.x & 63, E = p.E;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const int64_t s = p.off ? find_sequence(p.off, p.S, p.T, t) : 0;
  if (s < 0 || (p.off && t >= clamp_offset(p.off, s + 1, p.T))) return;
  const float n = static_cast<float>(tokens[s]), mean = n * p.k / E;
  const float factor = n > 0.0f ? dloss[s] * (static_cast<float>(E) / p.k) / n / n : 0.0f;
  float z[V], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    z[i] = e < E ? load_logit<BF16>(p.z, t * p.ldl + e) : -INFINITY;
    m = fmaxf(m, z[i]);
  }
  m = wave_max(m);
  float q[V], rest[V], c[V], sum = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    rest[i] = 0.0f;
    q[i] = z[i] == -INFINITY ? 0.0f : score<SIGMOID>(z[i], m, rest[i]);
    c[i] = e < E ? static_cast<float>(counts[s * E + e]) - mean : 0.0f;
    sum += q[i];
    dot += q[i] * c[i];
  }
  sum = wave_sum(sum);
  dot = wave_sum(dot);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    if (e >= E) continue;
    float d = z[i] == -INFINITY ? 0.0f : factor * (q[i] * inv) * (c[i] - dot * inv) * rest[i];
    const int64_t at = t * ldd + e;
    if (BF16) {
      uint16_t* o = static_cast<uint16_t*>(dz) + at;
      if (accumulate) d += bf16_to_f32(*o);
      *o = f32_to_bf16(d);
    } else {
      float* o = static_cast<float*>(dz) + at;
      if (accumulate) d += *o;
      *o = d;
    }
  }
}

int balance_check(int dtype, int64_t ldl, int64_t T, int32_t E, int32_t k, int score, const int32_t* off, int32_t S) {
  if (T < 0 || T > INT32_MAX || E <= 0 || E > kMaxE || k <= 0 || k > kMaxK || k > E || ldl < E) return MOE_ERR_SHAPE;
  if (S < 1 || S > (1 << 24)) return MOE_ERR_SHAPE;
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (!off && S != 1) return MOE_ERR_NULL;
  return MOE_OK;
}

}  // namespace

// The error word, and a slot of E share sums, E counts and a token count for each chunk and sequence.
size_t balance_ws_bytes(int64_t T, int64_t S, int E) {
  const int64_t chunks = (T + chunk_tokens(T) - 1) / chunk_tokens(T);
  return static_cast<size_t>(kHeader + ((chunks + S) * (2 * E + 1) * 4 + 255) / 256 * 256);
}

}  // namespace moe

#define MOE_BY_V(CALL, B, S)                                      \
  do {                                                            \
    if (E <= 64) CALL(B, S, 1);                                   \
    else if (E <= 128) CALL(B, S, 2);                             \
    else if (E <= 256) CALL(B, S, 4);                             \
    else if (E <= 512) CALL(B, S, 8);                             \
    else CALL(B, S, 16);                                          \
  } while (0)
#define MOE_BY_TYPE(CALL)                                         \
  do {                                                            \
    const bool sig = score == MOE_SCORE_SIGMOID;                  \
    if (logits_dtype == MOE_BF16) {                               \
      if (sig) MOE_BY_V(CALL, true, true); else MOE_BY_V(CALL, true, false);    \
    } else {                                                      \
      if (sig) MOE_BY_V(CALL, false, true); else MOE_BY_V(CALL, false, false);  \
    }                                                             \
  } while (0)

extern "C" int moe_balance_loss(const void* logits, int logits_dtype, int64_t ldl, const int32_t* expert_ids, int64_t T,
                                int32_t E, int32_t k, int score, const int32_t* seq_offsets, int32_t S, float* loss,
                                int32_t* counts, int32_t* tokens, void* ws, size_t ws_bytes, void* stream) {
  const int c = moe::balance_check(logits_dtype, ldl, T, E, k, score, seq_offsets, S);
  if (c != MOE_OK) return c;
  if (!loss || !counts || !tokens || (T > 0 && (!logits || !expert_ids))) return MOE_ERR_NULL;
  if (!ws || ws_bytes < moe::balance_ws_bytes(T, S, E)) return MOE_ERR_WORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t chunk = moe::chunk_tokens(T), chunks = moe_cdiv(T, chunk);
  const moe::BalanceArgs p{logits, ldl, expert_ids, T, E, k, seq_offsets, S,
                           reinterpret_cast<float*>(static_cast<char*>(ws) + moe::kHeader), static_cast<int32_t*>(ws)};
  if (chunks > 0) {
#define MOE_LOSS(B, S, V) moe::balance_kernel<B, S, V><<<static_cast<unsigned>(chunks), 256, 0, st>>>(p, chunk)
    MOE_BY_TYPE(MOE_LOSS);
#undef MOE_LOSS
    MOE_CHECK_LAUNCH();
  }
  moe::balance_join_kernel<<<static_cast<unsigned>(S < 65536 ? S : 65536), 256, 0, st>>>(p, chunk, chunks, loss, counts, tokens);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_balance_loss_backward(const void* logits, int logits_dtype, int64_t ldl, const int32_t* counts,
                                         const int32_t* tokens, const float* dloss, int64_t T, int32_t E, int32_t k, int score,
                                         const int32_t* seq_offsets, int32_t S, int accumulate, void* dlogits, int64_t ldd,
                                         void* stream) {
  const int c = moe::balance_check(logits_dtype, ldl, T, E, k, score, seq_offsets, S);
  if (c != MOE_OK) return c;
  if (ldd < E) return MOE_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !tokens || !dloss || !dlogits) return MOE_ERR_NULL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const moe::BalanceArgs p{logits, ldl, nullptr, T, E, k, seq_offsets, S, nullptr, nullptr};
  const unsigned grid = static_cast<unsigned>(moe_cdiv(T, 4));
#define MOE_BWD(B, S, V) moe::balance_bwd_kernel<B, S, V><<<grid, 256, 0, st>>>(p, counts, tokens, dloss, accumulate, dlogits, ldd)
  MOE_BY_TYPE(MOE_BWD);
#undef MOE_BWD
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
