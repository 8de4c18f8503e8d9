// moe_ffn_tokens: a whole gated expert layer for a few tokens,
//   out[t] = sum_j w[t, j] * ((silu(x[t] W0_e) * (x[t] W1_e)) Wo_e),  e = ids[t, j],
// in three kernels.  At these sizes the experts' weights are the traffic: each
// chosen expert's weights are read once, from e4m3 codes or 4-bit blocks, and
// converted on the way to the matrix cores, while the activations stay as
// they are (bfloat16 rows; the hidden values as two bfloat16 pieces, 16 bits
// of mantissa, since they are small next to the weights) -- nothing is
// quantized, and every sum's order is fixed, so a token's result does not
// depend on the others'.
//
// The first two form weights (16 output channels) times rows (16 slots) with
// v_mfma_f32_16x16x32_bf16, 32 channels a wave at a time (a unit):
//   1  16 hidden channels' a and b -> h = silu(a) * b
//   2  y[slot] of 32 output channels
// and the third adds each token's slots in slot order.
//
// Memory bounds it, then three launches and, in each, the routing, the first
// loads and the tail.  Weights once at 5.2 TB/s; a call among others, from
// Python; the first two kernels in the trace, and their rates:
//   one token of 7168, 8 e4m3 experts of 2048         68  67 us     40, 26 us  5.8, 4.6 TB/s
//   16 tokens of 2048, 8 of 64 4-bit experts of 768   27  51        28, 22     3.4, 2.2
//   64 such tokens in e4m3                            58  65 to 77  39, 25     5.1, 4.0
// (Where two figures are compared below, both are calls as a graph, measured
// side by side when the step was taken.)
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
constexpr int kHeader = 256;                       // workspace: error word

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
  uint16_t* h;                                     // [2][slots][I]: high and low pieces
  float* y;                                        // [slots][H]
};

constexpr int kRing = 4;                           // chunks of weights in LDS a wave
constexpr int kChunk = 4096;                       // 32 rows of 128 bytes
constexpr int kScales = 384;                       // a chunk's scales: 4-bit 32 rows of 3 dwords, e4m3 32 floats
constexpr int kRows = 16;                          // slots at a time
constexpr int kXBytes = 2 * kRows * (2048 + 16);  // both pieces of 16 rows' 1024 elements, the least that run_units stages

struct Lds {
  uint8_t w[kWaves][kRing][kChunk];
  uint8_t s[kWaves][kRing][kScales];
  uint8_t x[kXBytes];                              // rows of the slots at hand
  float red[kWaves][8][64];
  // the routing: every workgroup derives it for itself
  int16_t local[kMaxSlots];                        // local expert of a slot, or -1
  uint16_t met[kMaxLocalE], count[kMaxLocalE];     // the met experts, ascending, and their slots
  uint16_t list[kMaxSlots];                        // the slots of the expert at hand, ascending
  int n_met;
};
static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a CU");

__device__ void read_routing(const FfnArgs& p, Lds& sm) {
  const int tid = threadIdx.x, n = p.T * p.k;
  int* count = reinterpret_cast<int*>(sm.x);
  for (int e = tid; e < p.El; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int s = tid; s < n; s += kThreads) {
    const int id = p.ids[s];
    const int e = id >= p.g0 && id < p.g0 + p.El && id >= 0 && id < p.E ? id - p.g0 : -1;
    sm.local[s] = static_cast<int16_t>(e);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  if (tid < 64) {                                  // wave 0: compaction
    int at = 0;
    for (int b = 0; b < p.El; b += 64) {
      const int c = b + tid < p.El ? count[b + tid] : 0;
      const uint64_t mask = __ballot(c > 0);
      if (c > 0) {
        const int i = at + __popcll(mask & ((1ull << tid) - 1));
        sm.met[i] = static_cast<uint16_t>(b + tid);
        sm.count[i] = static_cast<uint16_t>(c);
      }
      at += __popcll(mask);
    }
    if (tid == 0) sm.n_met = at;
  }
  __syncthreads();
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8*)p));
}
// LDS through integer addresses: for a pointer into what the direct loads fill
// the compiler would wait for every load in flight before each read.
template <class T>
__device__ __forceinline__ T lds_read(uint32_t a) {
  return *(const __attribute__((address_space(3))) T*)(uintptr_t)(a);
}
template <class T>
__device__ __forceinline__ void lds_write(uint32_t a, T v) {
  *(__attribute__((address_space(3))) T*)(uintptr_t)(a) = v;
}
// s_waitcnt vmcnt(n) alone.
constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
__device__ __forceinline__ void order() { asm volatile("" ::: "memory"); }
// A barrier that leaves loads in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The slots of local expert e, ascending, into the list.  (Wave 0 scans in
// order, so the order does not depend on timing.)
__device__ void list_slots(const FfnArgs& p, Lds& sm, int e) {
  const int n = p.T * p.k, tid = threadIdx.x;
  if (tid < 64) {
    int at = 0;
    for (int b = 0; b < n; b += 64) {
      const bool in = b + tid < n && lds_read<int16_t>(lds_addr(sm.local + min(b + tid, n - 1))) == e;
      const uint64_t mask = __ballot(in);
      if (in) lds_write<uint16_t>(lds_addr(sm.list + at + __popcll(mask & ((1ull << tid) - 1))), static_cast<uint16_t>(b + tid));
      at += __popcll(mask);
    }
  }
}

// Eight e4m3 codes (two words) to bfloat16, exactly.
__device__ __forceinline__ bf8 bf16_of_e4m3(uint32_t a, uint32_t b) {
  const bf2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// Eight e2m1 codes (one word) times a power of two up to 2^125 to bfloat16,
// exactly (2^-127 and its half are subnormal, and kept); a scale that is NaN
// gives NaN for every code, 0 among them (measured on the device).
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

// The units of one call, in a run over the met experts, and this workgroup's
// part of them, in segments of one expert each.  A segment's units go to the
// four waves in turn, each wave a unit of its own; the one to three left over
// are formed by all four waves together, which split the contraction.  Which
// of the two a unit falls to depends on the other tokens' experts, and a
// token's result must not: either way chunk c of the contraction goes to sum
// c % 4 of four, which are added as (0 + 1) + (2 + 3).
struct Segment {
  int first, last, expert;                         // units; index of the met expert
  int full, jobs, passes;                          // units a wave of its own; jobs a pass; passes of 16 slots
};
__device__ __forceinline__ Segment segment_at(const Lds& sm, int u, int end, int units) {
  Segment s;
  s.first = u;
  s.expert = u / units;
  s.last = min(end, (s.expert + 1) * units);
  s.full = (s.last - u) / kWaves;
  s.jobs = s.full + (s.last - u) % kWaves;
  s.passes = (uniform(lds_read<uint16_t>(lds_addr(sm.count + s.expert))) + kRows - 1) / kRows;
  return s;
}
__device__ __forceinline__ int unit_of(const Segment& s, int job, int wave) {
  return job < s.full ? s.first + kWaves * job + wave : s.first + (kWaves - 1) * s.full + job;
}

// Weights of one matrix set: unit u of expert e is the 16 rows from row
// `row(u, 0)` and the 16 from `row(u, 1)`.
template <bool UP>
struct Weights {
  const uint8_t* w;
  const void* s;
  int64_t K, N;                                    // row length; rows an expert
  int kb, nb;
  __device__ __forceinline__ int64_t row(int u, int r) const {
    return UP ? r * (N / 2) + 16 * u : min(static_cast<int64_t>(32) * u + 16 * r, N - 16);
  }
};

// The chunks of weights that a wave loads, in the order it needs them, over
// all of the workgroup's segments: the loads run ahead of everything else.
template <bool MX4, bool UP>
struct Loader {
  static constexpr int kLoads = 4 + (MX4 ? 2 : 1); // loads a chunk
  const Weights<UP>& m;
  Lds& sm;
  Segment seg;
  int end, units, chunks, wave, lane;
  int block_len;                                   // e4m3: elements of a K block (32-bit: 64-bit divisions were most of the code)
  int pass, job, c, step, q;                       // q: chunks loaded so far
  bool more;
  const uint8_t *w0, *w1, *s0, *s1;                // of the job

  __device__ __forceinline__ Loader(const Weights<UP>& m, Lds& sm, int first, int end, int units, int wave, int lane)
      : m(m), sm(sm), end(end), units(units), wave(wave), lane(lane) {
    chunks = static_cast<int>((m.K / (MX4 ? 2 : 1) + 127) / 128);
    if constexpr (!MX4) block_len = static_cast<int>(m.K) / m.kb;
    q = 0;
    more = first < end;
    if (more) {
      seg = segment_at(sm, first, end, units);
      pass = job = 0;
      begin();
      settle();
    }
  }
  __device__ __forceinline__ void begin() {        // the first chunk of a job
    const bool own = job < seg.full;
    c = own ? 0 : wave;
    step = own ? 1 : kWaves;
    const int u = unit_of(seg, job, wave) - seg.expert * units;
    const int64_t e = uniform(lds_read<uint16_t>(lds_addr(sm.met + seg.expert)));
    const int64_t r0 = m.row(u, 0), r1 = m.row(u, 1), rowb = m.K / (MX4 ? 2 : 1);
    w0 = m.w + (e * m.N + r0) * rowb;
    w1 = m.w + (e * m.N + r1) * rowb;
    if constexpr (MX4) {
      s0 = static_cast<const uint8_t*>(m.s) + (e * m.N + r0) * (m.K / 32);
      s1 = static_cast<const uint8_t*>(m.s) + (e * m.N + r1) * (m.K / 32);
    } else {                                       // one K block's factors: a channel's own, or its column block's
      const float* s = static_cast<const float*>(m.s) + e * m.kb * m.nb;
      const int wide = static_cast<int>(m.N) / m.nb;
      s0 = reinterpret_cast<const uint8_t*>(s + static_cast<int>(r0) / wide);
      s1 = reinterpret_cast<const uint8_t*>(s + static_cast<int>(r1) / wide);
    }
  }
  __device__ __forceinline__ void settle() {       // (a short row may leave a wave without a chunk of a split unit)
    while (c >= chunks) {
      if (++job == seg.jobs) {
        job = 0;
        if (++pass == seg.passes) {
          pass = 0;
          if (seg.last >= end) {
            more = false;
            return;
          }
          seg = segment_at(sm, seg.last, end, units);
        }
      }
      begin();
    }
  }
  // AUX 2: not kept in the caches.  Weights that one pass reads are read once (one token e4m3 75 us instead of
  // 83, 64 tokens 69 instead of 77); those of an expert with more slots than a pass takes are read again.
  __device__ __forceinline__ void load() {
    if (seg.passes == 1)
      load<2>();
    else
      load<0>();
    ++q;
    c += step;
    settle();
  }
  template <int AUX>
  __device__ __forceinline__ void load() {
    const int slot = q % kRing, rowb = static_cast<int>(m.K / (MX4 ? 2 : 1));
    uint8_t* wd = sm.w[wave][slot];
    uint8_t* sd = sm.s[wave][slot];
    // rows of eight lanes; LDS piece s of row r holds the row's piece s ^ swz(r); pieces past the row: its last
    const int row = lane >> 3, sp = (lane & 7) ^ row;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = min(128 * c + 16 * (sp ^ (i & 1)), rowb - 16);
      __builtin_amdgcn_global_load_lds((i < 2 ? w0 : w1) + static_cast<uint32_t>((8 * (i & 1) + row) * rowb + b),
                                       (lds_void*)(wd + 1024 * i), 16, 0, AUX);
    }
    if constexpr (MX4) {                           // the three dwords that hold a row's eight scales
      const int kb = static_cast<int>(m.K / 32);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int idx = 64 * i + lane, r = idx / 3;
        const int b = min((((r & 15) * kb + 8 * c) & ~3) + 4 * (idx - 3 * r), 16 * kb - 4);
        if (idx < 96) __builtin_amdgcn_global_load_lds((r < 16 ? s0 : s1) + b, (lds_void*)(sd + 256 * i), 4, 0, 0);
      }
    } else {
      const int64_t block = static_cast<int64_t>(128 * c / block_len) * m.nb;
      const int ch = m.nb == m.N ? lane & 15 : 0;
      if (lane < 32) __builtin_amdgcn_global_load_lds((lane < 16 ? s0 : s1) + 4 * (block + ch), (lds_void*)sd, 4, 0, 0);
    }
  }
};

// Both kernels' loop over a workgroup's units.  rows(slot, piece) gives a
// slot's row (P pieces of the same values' significance, added up), and
// finish(unit, slot, live, acc, i0, ni) takes the sums: element i of block r
// is channel 4 (l/16) + i of slot l%16, valid for i0 <= i < i0 + ni.
//
// One workgroup of four waves a CU.  Weights come to LDS by direct loads of
// whole 128-byte lines, each wave its own, kRing chunks ahead and on across
// units and experts (16 KB a wave in flight).  Loaded to registers in the order
// the matrix cores want them, by many small workgroups that each wait for
// their own unit, the same layers took 113, 68 and 132 us where this took 83,
// 53 and 78.  The slots' rows are staged once an expert where they fit, else
// by parts of the contraction.
template <bool MX4, bool UP, int P, class Rows, class Finish>
__device__ __forceinline__ void run_units(const Weights<UP>& m, Lds& sm, const FfnArgs& p, int first, int end, int units,
                                          const Rows& rows, const Finish& finish) {
  using L = Loader<MX4, UP>;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), l15 = lane & 15, grp = lane >> 4;
  constexpr int CK = MX4 ? 256 : 128;              // elements a chunk
  const int K = static_cast<int>(m.K), kb = K / 32;
  L load(m, sm, first, end, units, wave, lane);
  const int chunks = static_cast<int>((m.K / (MX4 ? 2 : 1) + 127) / 128);
  for (int i = 0; i < kRing; ++i)
    if (load.more) load.load();
  int q = 0;                                       // chunks consumed
  const uint32_t wa0 = lds_addr(sm.w[wave]) + l15 * 128 + 16 * (grp ^ ((l15 & 7) ^ (l15 >> 3)));
  const uint32_t sa0 = lds_addr(sm.s[wave]) + (MX4 ? l15 * 12 + grp + ((l15 * kb) & 3) : 16 * grp);

  for (int at = first; at < end;) {
    const Segment seg = segment_at(sm, at, end, units);
    at = seg.last;
    const int e = uniform(lds_read<uint16_t>(lds_addr(sm.met + seg.expert)));
    const int ns = uniform(lds_read<uint16_t>(lds_addr(sm.count + seg.expert)));
    lds_barrier();                                 // the last segment's list is read
    list_slots(p, sm, e);
    lds_barrier();
    for (int pass = 0; pass < seg.passes; ++pass) {
      const int n = min(ns - kRows * pass, kRows);
      // elements of a row that fit, in whole chunks of all four waves
      const int fit = (kXBytes / (n * P) - 16) / 2, KC = K <= fit ? K : fit / (kWaves * CK) * (kWaves * CK);
      const uint32_t pitch = 2 * KC + 16;          // (rows one 16-byte bank group apart)
      const int my = l15 < n ? l15 : 0;
      const uint32_t xa0 = lds_addr(sm.x) + my * P * pitch + (MX4 ? 64 : 32) * grp;
      const int slot = lds_read<uint16_t>(lds_addr(sm.list + kRows * pass + my));
      auto stage = [&](int k0) {
        lds_barrier();                             // the last rows are read
        const int len = min(K - k0, KC) / 8;       // 16-byte pieces
        for (int i = wave; i < n * P; i += kWaves) {
          const uint16_t* src = rows(uniform(lds_read<uint16_t>(lds_addr(sm.list + kRows * pass + i / P))), i % P) + k0;
          for (int b = 0; b < len; b += 64)
            if (b + lane < len)
              __builtin_amdgcn_global_load_lds(src + 8 * (b + lane), (lds_void*)(sm.x + i * pitch + 16 * b), 16, 0, 0);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        lds_barrier();
      };
      if (KC == K) stage(0);
      for (int job = 0; job < seg.jobs; ++job) {
        const bool own = job < seg.full;
        v4f sums[kWaves][2];                       // (of a split unit each wave fills its first)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sums[w][0] = sums[w][1] = v4f{0.f, 0.f, 0.f, 0.f};
        int c = own ? 0 : wave;
        for (int k0 = 0; k0 < K; k0 += KC) {
          if (KC < K) stage(k0);
          const int stop = min((k0 + KC + CK - 1) / CK, chunks);
          auto chunk = [&](int c, v4f(&acc)[2]) __attribute__((always_inline)) {
            const int slot_at = q % kRing;
            if (load.more)                         // then all kRing - 1 later chunks are in flight, in order
              __builtin_amdgcn_s_waitcnt(waitcnt_vm((kRing - 1) * L::kLoads));
            else
              __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
            order();
            const uint32_t wa = wa0 + slot_at * kChunk, sa = sa0 + slot_at * kScales, xa = xa0 + 2 * (CK * c - k0);
            u4 w[2][2];
            float sc[2][MX4 ? 2 : 4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              w[r][0] = lds_read<u4>(wa + 2048 * r);
              w[r][1] = lds_read<u4>((wa ^ 64) + 2048 * r);
              if constexpr (MX4) {
                sc[r][0] = mx4::scale_value(lds_read<uint8_t>(sa + 192 * r));
                sc[r][1] = mx4::scale_value(lds_read<uint8_t>(sa + 192 * r + 4));
              } else {
                const v4f v = lds_read<v4f>(sa + 64 * r);
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[r][i] = v[i];
              }
            }
            constexpr int NX = MX4 ? 4 : 2;        // groups of 8 elements a piece of 16 bytes
            u4 xv[P][2][NX];
#pragma unroll
            for (int b = 0; b < P; ++b)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < NX; ++u) xv[b][h][u] = lds_read<u4>(xa + b * pitch + CK * h + 16 * u);
            // the chunk's slot is read: load it again
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (load.more) load.load();
            order();
            ++q;
            if (CK * c + CK > K) {                 // pieces past the row: nothing
              const u4 z = {0, 0, 0, 0};
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (CK * c + (CK / 8) * (grp + 4 * h) >= K) {
                  w[0][h] = w[1][h] = z;
#pragma unroll
                  for (int b = 0; b < P; ++b)
#pragma unroll
                    for (int u = 0; u < NX; ++u) xv[b][h][u] = z;
                  if constexpr (MX4) sc[0][h] = sc[1][h] = 1.0f;
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (MX4) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int u = 0; u < 4; ++u) {
                    const bf8 wv = bf16_of_e2m1(w[r][h][u], sc[r][h]);
#pragma unroll
                    for (int b = 0; b < P; ++b) acc[r] = mfma_bf16(wv, __builtin_bit_cast(bf8, xv[b][h][u]), acc[r]);
                  }
              } else {                             // a chunk lies in one K block: its scales multiply the chunk's sum
                v4f part = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const bf8 wv = bf16_of_e4m3(w[r][h][2 * u], w[r][h][2 * u + 1]);
#pragma unroll
                    for (int b = 0; b < P; ++b) part = mfma_bf16(wv, __builtin_bit_cast(bf8, xv[b][h][u]), part);
                  }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(sc[r][i], part[i], acc[r][i]);
              }
            }
          };
          // Four chunks a turn (one, where the unit is split; a part of the contraction ends at a multiple of four chunks,
          // or at its end): the sums keep their registers.  Moved round by one a chunk, one copy of the code, the layer
          // of 64 tokens took 86 us instead of 81.
#pragma clang loop unroll(disable)
          for (; c < stop; c += kWaves) {
            if constexpr (MX4) {                   // in the accumulators' own registers (else moved there and back each turn: 56.5 us for 54.7)
#pragma unroll
              for (int w = 0; w < kWaves; ++w) asm volatile("" : "+a"(sums[w][0]), "+a"(sums[w][1]));
            }
            chunk(c, sums[0]);
            if (!own) continue;
            if (c + 1 < stop) chunk(c + 1, sums[1]);
            if (c + 2 < stop) chunk(c + 2, sums[2]);
            if (c + 3 < stop) chunk(c + 3, sums[3]);
          }
        }
        const int unit = unit_of(seg, job, wave) - seg.expert * units;
        if (own) {
          const v4f sum[2] = {(sums[0][0] + sums[1][0]) + (sums[2][0] + sums[3][0]),
                              (sums[0][1] + sums[1][1]) + (sums[2][1] + sums[3][1])};
          finish(unit, slot, l15 < n, sum, 0, 4);
        } else {                                   // wave w finishes element w of both blocks
          lds_barrier();
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) lds_write<float>(lds_addr(&sm.red[wave][4 * r + i][lane]), sums[0][r][i]);
          lds_barrier();
          v4f sum[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float t[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) t[w] = lds_read<float>(lds_addr(&sm.red[w][4 * r + wave][lane]));
            const float v = (t[0] + t[1]) + (t[2] + t[3]);
            sum[r] = v4f{v, v, v, v};
          }
          finish(unit, slot, l15 < n, sum, wave, 1);
        }
      }
    }
  }
}

// This workgroup's units: a run.
__device__ __forceinline__ int share(int64_t n, unsigned b) { return static_cast<int>(n * b / gridDim.x); }

template <bool MX4>
__global__ __launch_bounds__(kThreads) void ffn_up_kernel(const FfnArgs p) {
  __shared__ __attribute__((aligned(1024))) Lds sm;
  read_routing(p, sm);
  const int64_t H = p.H, I = p.I, slots = static_cast<int64_t>(p.T) * p.k;
  const int units = static_cast<int>(I / 16);
  const int64_t n = static_cast<int64_t>(uniform(sm.n_met)) * units;
  const int grp = (threadIdx.x & 63) >> 4;
  const Weights<true> m{p.w01, p.s01, H, 2 * I, p.kb01, p.nb01};
  run_units<MX4, true, 1>(
      m, sm, p, share(n, blockIdx.x), share(n, blockIdx.x + 1), units,
      [&](int slot, int) { return p.x + static_cast<int64_t>(slot / p.k) * p.ldx; },
      [&](int unit, int slot, bool live, const v4f (&acc)[2], int i0, int ni) {
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = acc[0][i], hv = a / (1.0f + expf(-a)) * acc[1][i];
          hi[i] = f32_to_bf16(hv);
          const float rest = hv - bf16_to_f32(hi[i]);   // not finite: the high piece alone says so
          lo[i] = fabsf(rest) < INFINITY ? f32_to_bf16(rest) : 0;
        }
        if (!live) return;
        uint16_t* d = p.h + static_cast<int64_t>(slot) * I + 16 * unit + 4 * grp;
        if (ni == 4) {
          __builtin_memcpy(__builtin_assume_aligned(d, 8), hi, 8);
          __builtin_memcpy(__builtin_assume_aligned(d + slots * I, 8), lo, 8);
        } else {                                   // (all four are the same)
          d[i0] = hi[0];
          d[slots * I + i0] = lo[0];
        }
      });
}

template <bool MX4>
__global__ __launch_bounds__(kThreads) void ffn_down_kernel(const FfnArgs p) {
  __shared__ __attribute__((aligned(1024))) Lds sm;
  read_routing(p, sm);
  const int64_t H = p.H, I = p.I, slots = static_cast<int64_t>(p.T) * p.k;
  const int units = static_cast<int>((H + 31) / 32);
  const int64_t n = static_cast<int64_t>(uniform(sm.n_met)) * units;
  const int grp = (threadIdx.x & 63) >> 4;
  const Weights<false> m{p.wo, p.so, I, H, p.kbo, p.nbo};
  run_units<MX4, false, 2>(
      m, sm, p, share(n, blockIdx.x), share(n, blockIdx.x + 1), units,
      [&](int slot, int piece) { return p.h + (piece * slots + slot) * I; },
      [&](int unit, int slot, bool live, const v4f (&acc)[2], int i0, int ni) {
        if (!live) return;
        float* d = p.y + static_cast<int64_t>(slot) * H + 32 * static_cast<int64_t>(unit) + 4 * grp;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (32 * static_cast<int64_t>(unit) + 16 * r >= H) continue;
          if (ni == 4)
            *reinterpret_cast<v4f*>(d + 16 * r) = acc[r];
          else
            d[16 * r + i0] = acc[r][0];
        }
      });
}

// The output: each token's slots, in slot order; a lane four columns.  (A kernel of its own: left to the workgroup
// that finishes a column block last, it falls to the few that end last of all.)
__global__ __launch_bounds__(kThreads) void ffn_combine_kernel(const FfnArgs p) {
  const int64_t quads = p.H / 4, n = p.T * quads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int t = static_cast<int>(i / quads);
    const int64_t c = 4 * (i - t * quads);
    v4f v = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < p.k; j0 += 4) {          // four slots' loads at a time
      v4f y[4];
      float w[4];
      bool in[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = t * p.k + min(j0 + j, p.k - 1), id = p.ids[s];
        in[j] = j0 + j < p.k && id >= 0 && id < p.E && id >= p.g0 && id < p.g0 + p.El;
        w[j] = p.tw[s];
        if (c == 0 && (id < 0 || id >= p.E)) raise_error(p.err, MOE_DEVERR_EXPERT_ID);
        y[j] = *reinterpret_cast<const v4f*>(p.y + static_cast<int64_t>(s) * p.H + c);     // (unused where no expert wrote it)
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (in[j]) v[q] = fmaf(w[j], y[j][q], v[q]);
    }
    if (p.out_bf16) {
      const uint32_t o[2] = {f32_to_bf16(v[0]) | static_cast<uint32_t>(f32_to_bf16(v[1])) << 16,
                             f32_to_bf16(v[2]) | static_cast<uint32_t>(f32_to_bf16(v[3])) << 16};
      __builtin_memcpy(__builtin_assume_aligned(static_cast<uint16_t*>(p.out) + t * p.H + c, 8), o, 8);
    } else {
      *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + t * p.H + c) = v;
    }
  }
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Error word, the hidden pieces, the slots' outputs.
size_t ffn_tokens_ws_bytes(int64_t slots, int64_t H, int64_t I) {
  return static_cast<size_t>(kHeader + align256(4 * slots * I) + align256(4 * slots * H));
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
  if (E <= 0 || E > 1024 || group_offset < 0 || num_local_experts < 0 || group_offset > E - num_local_experts)
    return MOE_ERR_SHAPE;
  if (H > (int64_t{1} << 20) || I > (int64_t{1} << 20)) return MOE_ERR_SHAPE;   // units, and offsets in 16 rows, stay below 2^31
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
  if (reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(out) % 16 || reinterpret_cast<uintptr_t>(w01) % 16 || reinterpret_cast<uintptr_t>(wo) % 16 ||
      reinterpret_cast<uintptr_t>(w01_scale) % 4 || reinterpret_cast<uintptr_t>(wo_scale) % 4)
    return MOE_ERR_SHAPE;
  const int64_t slots = T * k;
  if (!ws || ws_bytes < ffn_tokens_ws_bytes(slots, H, I)) return MOE_ERR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  const int64_t h_off = kHeader, y_off = h_off + align256(4 * slots * I);
  const FfnArgs p{static_cast<const uint16_t*>(x), ldx, expert_ids, topk_weights, static_cast<int>(T), k, H, I, E,
                  group_offset, num_local_experts, w01, w01_scale, kb01, nb01, wo, wo_scale, kbo, nbo, out,
                  out_dtype == MOE_BF16, reinterpret_cast<int32_t*>(base),
                  reinterpret_cast<uint16_t*>(base + h_off), reinterpret_cast<float*>(base + y_off)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t most = slots < num_local_experts ? slots : num_local_experts;      // experts that can be met
  const int64_t cap = tile::num_cus();
  const int64_t up = most * (I / 16), down = most * moe_cdiv(H, 32), quads = moe_cdiv(T * (H / 4), kThreads);
  const unsigned gu = static_cast<unsigned>(up < cap ? up : cap), gd = static_cast<unsigned>(down < cap ? down : cap);
  if (most > 0) {
    if (mx)
      ffn_up_kernel<true><<<gu, kThreads, 0, st>>>(p);
    else
      ffn_up_kernel<false><<<gu, kThreads, 0, st>>>(p);
    MOE_CHECK_LAUNCH();
    if (mx)
      ffn_down_kernel<true><<<gd, kThreads, 0, st>>>(p);
    else
      ffn_down_kernel<false><<<gd, kThreads, 0, st>>>(p);
    MOE_CHECK_LAUNCH();
  }
  ffn_combine_kernel<<<static_cast<unsigned>(quads < 2 * cap ? quads : 2 * cap), kThreads, 0, st>>>(p);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
