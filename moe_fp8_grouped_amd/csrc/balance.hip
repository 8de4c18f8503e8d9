// moe_balance_loss / moe_balance_loss_backward: how evenly a router spreads
// its tokens, per sequence, and the gradient to the logits.  With the shares
// p_t of a token's scores over the experts in service, n tokens that have one,
// and c[e] choices of expert e in the sequence:
//   loss = E / (k n^2) sum_e c[e] sum_t p[t, e]
//   dz[t, e] = dloss E / (k n^2) p_e (c[e] - sum_f c[f] p_f) r_e
// r = 1 for softmax shares, 1 - sigmoid(z) for normalised sigmoids.
// Launches and a chunk's chain of loads and sums bound the loss, not its bytes: 8192
// tokens of 256 experts in bf16 take 16 us, 9.4 for the chunks (0.5 TB/s) and 6.8 to
// join them; the gradient of 32768 tokens of 64 experts 7.5 us (2.2 TB/s).
#include "wave_common.hpp"

namespace moe {
namespace {

constexpr int kMaxE = 1024, kMaxK = 64;
constexpr float kOut = -1e30f;               // a logit at or below it, or NaN, takes its expert out
constexpr int64_t kHeader = 256;             // workspace: error word
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kChunk = 64;                   // tokens of a workgroup of the forward pass, at least: four a wave

// G lanes (16 or the whole wave) share a row, lane `sub` of them holds experts 4 G i + 4 sub .. + 3 for i < V.
template <bool BF16, int G, int V>
struct Row {
  float z[V][4];

  // `wide`: whole, aligned vectors of four
  __device__ __forceinline__ void load(const void* p, int64_t at, int E, int sub, bool wide) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 4 * G * i + 4 * sub;
#pragma unroll
      for (int c = 0; c < 4; ++c) z[i][c] = -INFINITY;
      if (wide && e < E) {
        if (BF16) {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at + e);
          z[i][0] = __uint_as_float(v.x << 16);
          z[i][1] = __uint_as_float(v.x & 0xffff0000u);
          z[i][2] = __uint_as_float(v.y << 16);
          z[i][3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
          const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + e);
          z[i][0] = v.x;
          z[i][1] = v.y;
          z[i][2] = v.z;
          z[i][3] = v.w;
        }
      } else if (!wide) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e + c < E) z[i][c] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[at + e + c]) : static_cast<const float*>(p)[at + e + c];
      }
    }
  }
  __device__ __forceinline__ float mask() {            // experts taken out; the largest logit left
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        z[i][c] = z[i][c] > kOut ? z[i][c] : -INFINITY;
        m = fmaxf(m, z[i][c]);
      }
    return G == 16 ? row_max(m) : max_of(m);
  }
};
template <int G>
__device__ __forceinline__ float over_row(float v) {
  return G == 16 ? row_sum(v) : sum_of(v);
}

// exp(x), x <= 0, within 1.5 units in the last place (0 below 2^-126): x log2 e as a sum of two floats, the power of two of the
// larger by the hardware, corrected by 1 + ln 2 times the smaller.  (The power of the rounded product alone is off by up
// to 58 units of 2^-24 at x = -84.  With expf and IEEE quotients the loss of 8192 tokens of 256 experts takes 17.5 us where this takes
// 16.8, the gradient of 32768 sigmoid rows of 64 experts 9.2 where this takes 7.5; with the rounded product 16.0 and 7.3.)
__device__ __forceinline__ float exp_of(float x) {
  x = fmaxf(x, -150.0f);
  const float h = x * 0x1.715476p+0f;
  const float l = fmaf(x, 0x1.4ae0cp-26f, fmaf(x, 0x1.715476p+0f, -h));
  const float e = __builtin_amdgcn_exp2f(h);
  return fmaf(e, l * 0x1.62e43p-1f, e);
}
// 1 / x for x from 1/2 to 2^11, within half a unit (and 2^-22 of one): the hardware's estimate and one step of Newton's.
__device__ __forceinline__ float inverse_of(float x) {
  const float y = __builtin_amdgcn_rcpf(x);
  return fmaf(fmaf(-x, y, 1.0f), y, y);
}

// A score up to a factor common to the row, with m its largest logit: exp(z - m), or
// sigmoid(z) / exp(min(m, 0)) = exp(min(z, 0) - min(m, 0)) / (1 + exp(-|z|)),
// which stays in range where every sigmoid of the row is below it.  0 for an
// expert taken out.
template <bool SIGMOID>
__device__ __forceinline__ float score(float z, float m, float& rest) {
  if (z == -INFINITY) return 0.0f;
  if constexpr (SIGMOID) {
    const float e = exp_of(-fabsf(z)), d = inverse_of(1.0f + e);
    rest = z < 0.0f ? d : e * d;
    return (z < 0.0f ? exp_of(z - fminf(m, 0.0f)) : 1.0f) * d;
  } else {
    rest = 1.0f;
    return exp_of(z - m);
  }
}

__device__ __forceinline__ int clamp_offset(const int32_t* off, int64_t s, int64_t T) {
  return static_cast<int>(min(static_cast<int64_t>(max(off[s], 0)), T));
}

// The last sequence that starts at or before token t, or -1: sixty-four candidates at a time, one a lane.
__device__ __forceinline__ int find_sequence(const int32_t* off, int S, int64_t T, int64_t t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = S;
  while (true) {
    const int stride = (n + 63) / 64, at = lane * stride;
    const int c = __popcll(__ballot(at < n && clamp_offset(off, lo + min(at, n - 1), T) <= t));
    if (stride == 1) return lo + c - 1;
    if (c == 0) return lo - 1;
    lo += (c - 1) * stride;
    n = min(stride, n - (c - 1) * stride);
  }
}

// Tokens of one workgroup of the forward pass.
__host__ __device__ inline int64_t chunk_tokens(int64_t T) {
  const int64_t c = (T + 511) / 512;
  return c < kChunk ? kChunk : c;
}

struct BalanceArgs {
  const void* z;
  int64_t ldl;
  const int32_t* ids;
  int64_t T;
  int E, k;
  const int32_t* off;
  int S;
  bool wide;
  float* part;                               // [chunks + S][E] share sums, then the same of counts, then of tokens
  int32_t* err;
};

// A workgroup takes a run of tokens, and leaves the sums of each sequence that
// it meets in a slot of its own: chunk + sequence.  (From one piece to the next the
// chunk or the sequence grows, so no two pieces share a slot, and a sequence's
// slots are a run.)
template <bool BF16, bool SIGMOID, int G, int V>
__global__ __launch_bounds__(kThreads) void balance_kernel(const BalanceArgs p, int64_t chunk) {
  constexpr int PER = 64 / G, U = G == 16 ? 1 : V >= 2 ? 2 : 4;          // rows a wave at a time, and how often before they are used
  __shared__ __attribute__((aligned(16))) float sums[kWaves][4 * G * V];
  __shared__ int counts[4 * G * V], tokens;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane & (G - 1), E = p.E;
  const int64_t slots = gridDim.x + static_cast<int64_t>(p.S);
  float* part = p.part;
  int32_t* cpart = reinterpret_cast<int32_t*>(part + slots * E);
  int32_t* npart = cpart + slots * E;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk, t1 = min(t0 + chunk, p.T);
  int s = p.off ? find_sequence(p.off, p.S, p.T, t0) : 0;
  int64_t t = t0;
  if (s < 0) {
    s = 0;
    t = max(t0, static_cast<int64_t>(clamp_offset(p.off, 0, p.T)));
  }
  for (; s < p.S && t < t1; ++s) {
    const int64_t end = p.off ? min(static_cast<int64_t>(clamp_offset(p.off, s + 1, p.T)), t1) : t1;
    if (end <= t) continue;
    for (int i = tid; i < E; i += kThreads) counts[i] = 0;
    if (tid == 0) tokens = 0;
    __syncthreads();
    float acc[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
    int n = 0;
    for (int64_t r0 = t + wave * PER * U; r0 < end; r0 += kWaves * PER * U) {
      Row<BF16, G, V> row[U];
      const int rows = static_cast<int>(min(end - r0, static_cast<int64_t>(PER * U)));
      // the first 64 choices and their logits beside the rows, any more behind them
      const int id0 = lane < rows * p.k ? p.ids[r0 * p.k + lane] : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) row[u].load(p.z, min(r0 + u * PER + lane / G, end - 1) * p.ldl, E, sub, p.wide);
      auto logit = [&](int j, int id) {
        const int64_t at = (r0 + j / p.k) * p.ldl + id;
        return BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.z)[at]) : static_cast<const float*>(p.z)[at];
      };
      const bool in0 = id0 >= 0 && id0 < E;
      const float z0 = in0 ? logit(lane, id0) : -INFINITY;
      for (int j = 64 + lane; j < rows * p.k; j += 64) {
        const int id = p.ids[r0 * p.k + j];
        if (id >= 0 && id < E && logit(j, id) > kOut) atomicAdd(&counts[id], 1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float m = row[u].mask();
        if (m == -INFINITY || u * PER + lane / G >= rows) continue;      // a padded token, or none
        float q[V][4], sum = 0.0f, rest;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            q[i][c] = score<SIGMOID>(row[u].z[i][c], m, rest);
            sum += q[i][c];
          }
        const float inv = inverse_of(over_row<G>(sum));
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] = fmaf(q[i][c], inv, acc[i][c]);
        ++n;
      }
      if (z0 > kOut) atomicAdd(&counts[id0], 1);
    }
    if (sub == 0 && n) atomicAdd(&tokens, n);
    // the sums of the waves, in order (of a wave's rows of lanes first)
    const int64_t slot = blockIdx.x + static_cast<int64_t>(s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (G == 16)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[i][c] += __shfl_xor(acc[i][c], 16, 64);
          acc[i][c] += __shfl_xor(acc[i][c], 32, 64);
        }
      if (lane < G) *reinterpret_cast<float4*>(&sums[wave][4 * G * i + 4 * sub]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    }
    __syncthreads();
    if (tid < E) {                           // (E <= kThreads)
      float total = 0.0f;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) total += sums[q][tid];
      part[slot * E + tid] = total;
      cpart[slot * E + tid] = counts[tid];
    }
    if (tid == 0) npart[slot] = tokens;
    __syncthreads();
    t = end;
  }
}

// A workgroup a sequence: its slots' sums, each thread's run of them in order and the threads' in order, and the loss.
__global__ __launch_bounds__(kThreads) void balance_join_kernel(const BalanceArgs p, int64_t chunk, int64_t chunks, float* __restrict__ loss,
                                                                int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
  __shared__ float sums[kThreads];
  __shared__ int cs[kThreads], n_tokens;
  __shared__ float red[kWaves];
  const int tid = threadIdx.x, E = p.E;
  const int64_t slots = chunks + p.S;
  const float* part = p.part;
  const int32_t* cpart = reinterpret_cast<const int32_t*>(part + slots * E);
  const int32_t* npart = cpart + slots * E;
  const int parts = kThreads / E, mine = tid / E, x = tid - mine * E;    // (E <= kThreads)
  for (int64_t s = blockIdx.x; s < p.S; s += gridDim.x) {
    int64_t b = 0, e = p.T;
    if (p.off) {
      const int32_t lo = p.off[s], hi = p.off[s + 1];
      if (tid == 0 && (lo < 0 || hi < lo || hi > p.T)) raise_error(p.err, MOE_DEVERR_SEQUENCE);
      b = clamp_offset(p.off, s, p.T);
      e = clamp_offset(p.off, s + 1, p.T);
    }
    const int64_t first = b / chunk + s, count = e > b ? (e - 1) / chunk + s - first + 1 : 0;
    if (tid == 0) n_tokens = 0;
    float sum = 0.0f;
    int c = 0;
    if (mine < parts) {
      const int64_t per = (count + parts - 1) / parts, to = min((mine + 1) * per, count);
#pragma unroll 8
      for (int64_t i = mine * per; i < to; ++i) {
        sum += part[(first + i) * E + x];
        c += cpart[(first + i) * E + x];
      }
    }
    sums[tid] = sum;
    cs[tid] = c;
    __syncthreads();
    int n = 0;
    for (int64_t i = tid; i < count; i += kThreads) n += npart[first + i];
    if (n) atomicAdd(&n_tokens, n);
    float dot = 0.0f;
    if (tid < E) {
      for (int i = 1; i < parts; ++i) {
        sum += sums[i * E + tid];
        c += cs[i * E + tid];
      }
      counts[s * E + tid] = c;
      dot = static_cast<float>(c) * sum;
    }
    dot = sum_of(dot);
    if ((tid & 63) == 0) red[tid >> 6] = dot;
    __syncthreads();
    if (tid == 0) {
      float all = 0.0f;
      for (int i = 0; i < kWaves; ++i) all += red[i];
      tokens[s] = n_tokens;
      const double d = static_cast<double>(n_tokens);
      loss[s] = n_tokens > 0 ? static_cast<float>(static_cast<double>(all) * E / (p.k * d * d)) : 0.0f;
    }
    __syncthreads();
  }
}

// The gradient, G lanes a token.  The counts enter less their mean, which the
// gradient does not see (the shares sum to 1) and the differences keep their
// digits by.
template <bool BF16, bool SIGMOID, int G, int V>
__global__ __launch_bounds__(256) void balance_bwd_kernel(const BalanceArgs p, const int32_t* __restrict__ counts,
                                                          const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                                                          int accumulate, void* __restrict__ dz, int64_t ldd) {
  constexpr int PER = 64 / G;
  const int lane = threadIdx.x & 63, sub = lane & (G - 1), E = p.E;
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6)) * PER; r0 < p.T; r0 += static_cast<int64_t>(gridDim.x) * 4 * PER) {
    const int64_t t = r0 + lane / G, tc = min(t, p.T - 1);               // (past the last token: its copy, not stored)
    Row<BF16, G, V> row, old;
    row.load(p.z, tc * p.ldl, E, sub, p.wide);
    if (accumulate) old.load(dz, tc * ldd, E, sub, p.wide);
    int s = 0;
    if (p.off) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int f = find_sequence(p.off, p.S, p.T, min(r0 + j, p.T - 1));
        if (lane / G == j) s = f;
      }
    }
    const bool in = t < p.T && s >= 0 && !(p.off && t >= clamp_offset(p.off, max(s, 0) + 1, p.T));
    s = max(s, 0);
    const float n = static_cast<float>(tokens[s]), mean = n * p.k / E;
    const float factor = n > 0.0f ? dloss[s] * (static_cast<float>(E) / p.k) / n / n : 0.0f;
    float c[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 4 * G * i + 4 * sub;
      const int32_t* at = counts + static_cast<int64_t>(s) * E + e;
      int4 v = make_int4(0, 0, 0, 0);
      if (e + 3 < E && E % 4 == 0 && (reinterpret_cast<uintptr_t>(counts) & 15) == 0) {
        v = *reinterpret_cast<const int4*>(at);
      } else {
        if (e < E) v.x = at[0];
        if (e + 1 < E) v.y = at[1];
        if (e + 2 < E) v.z = at[2];
        if (e + 3 < E) v.w = at[3];
      }
      c[i][0] = static_cast<float>(v.x) - mean;
      c[i][1] = static_cast<float>(v.y) - mean;
      c[i][2] = static_cast<float>(v.z) - mean;
      c[i][3] = static_cast<float>(v.w) - mean;
    }
    const float m = row.mask();
    float q[V][4], rest[V][4], sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        rest[i][j] = 0.0f;
        q[i][j] = score<SIGMOID>(row.z[i][j], m, rest[i][j]);
        sum += q[i][j];
        dot += q[i][j] * c[i][j];
      }
    sum = over_row<G>(sum);
    dot = over_row<G>(dot);
    const float inv = sum > 0.0f ? inverse_of(sum) : 0.0f;
    if (!in) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 4 * G * i + 4 * sub;
      if (e >= E) continue;
      float d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = factor * (q[i][j] * inv) * (c[i][j] - dot * inv) * rest[i][j];
        if (accumulate) d[j] += old.z[i][j];
      }
      const int64_t at = t * ldd + e;
      if (p.wide) {
        if (BF16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dz) + at) =
              make_uint2(f32_to_bf16(d[0]) | static_cast<uint32_t>(f32_to_bf16(d[1])) << 16,
                         f32_to_bf16(d[2]) | static_cast<uint32_t>(f32_to_bf16(d[3])) << 16);
        else
          *reinterpret_cast<float4*>(static_cast<float*>(dz) + at) = make_float4(d[0], d[1], d[2], d[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (e + j >= E) continue;
          if (BF16)
            static_cast<uint16_t*>(dz)[at + j] = f32_to_bf16(d[j]);
          else
            static_cast<float*>(dz)[at + j] = d[j];
        }
      }
    }
  }
}

// Whole, aligned vectors of four logits.
bool four(const void* p, int64_t ld, int E, int dtype) {
  const uintptr_t size = dtype == MOE_BF16 ? 2 : 4;
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld | E) * size) % (4 * size) == 0;
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

// Sixteen lanes a row up to 128 experts, the whole wave above.  Loss and gradient of 8192 tokens in 5 sequences as graphs, us: 64 experts
// 12.1 and 4.4 (a wave a row 15.2 and 5.4), 128 experts 14.1 and 5.2 (16.1 and 5.7), 256 experts 16.8 and 6.1 (sixteen lanes
// 17.0 and 7.1); of 32768 tokens, 64 experts, 14.7 and 7.1 (18.8 and 13.7).
#define MOE_BY_V(CALL, B, S)                                      \
  do {                                                            \
    if (E <= 64) CALL(B, S, 16, 1);                               \
    else if (E <= 128) CALL(B, S, 16, 2);                         \
    else if (E <= 256) CALL(B, S, 64, 1);                         \
    else if (E <= 512) CALL(B, S, 64, 2);                         \
    else CALL(B, S, 64, 4);                                       \
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
  const moe::BalanceArgs p{logits, ldl, expert_ids, T, E, k, seq_offsets, S, moe::four(logits, ldl, E, logits_dtype),
                           reinterpret_cast<float*>(static_cast<char*>(ws) + moe::kHeader), static_cast<int32_t*>(ws)};
  if (chunks > 0) {
#define MOE_LOSS(B, S, G, V) moe::balance_kernel<B, S, G, V><<<static_cast<unsigned>(chunks), moe::kThreads, 0, st>>>(p, chunk)
    MOE_BY_TYPE(MOE_LOSS);
#undef MOE_LOSS
    MOE_CHECK_LAUNCH();
  }
  moe::balance_join_kernel<<<static_cast<unsigned>(S < 65536 ? S : 65536), moe::kThreads, 0, st>>>(p, chunk, chunks, loss, counts, tokens);
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
  const bool wide = moe::four(logits, ldl, E, logits_dtype) && moe::four(dlogits, ldd, E, logits_dtype);
  const moe::BalanceArgs p{logits, ldl, nullptr, T, E, k, seq_offsets, S, wide, nullptr, nullptr};
  const int64_t groups = moe_cdiv(T, E <= 128 ? 16 : 4);
  const unsigned grid = static_cast<unsigned>(groups < 65536 ? groups : 65536);
#define MOE_BWD(B, S, G, V) moe::balance_bwd_kernel<B, S, G, V><<<grid, 256, 0, st>>>(p, counts, tokens, dloss, accumulate, dlogits, ldd)
  MOE_BY_TYPE(MOE_BWD);
#undef MOE_BWD
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
