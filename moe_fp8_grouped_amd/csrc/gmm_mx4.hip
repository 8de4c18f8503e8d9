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
#include <type_traits>

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

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kFrags = 8;                        // row blocks of 16 a tile holds at most
constexpr int kRows = 16 * kFrags;
constexpr int kStages = 3;
constexpr int kStageBytes = kRows * 128;
constexpr int kPitch = 20;                       // LDS bytes a row of one scale window: 16 blocks, at any alignment
constexpr int kDesc = 64;                        // tiles decoded at a time

// Slot of 16-byte chunk c of staged row r: c ^ swz(r).  Eight consecutive rows
// use eight slots, so a fragment read (16 rows, served 8 lanes at a time) is
// free of bank conflicts.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// No memory access crosses: the order of the loads below is what the waits count.
__device__ __forceinline__ void order() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ void step_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A lane number that the compiler cannot carry from one use to the next: what
// follows from it is formed again where it is needed instead of being held in
// registers through the loop.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8*)p));
}

// Buffer over `bytes` bytes from p (uniform): loads take a lane offset and a
// uniform one, so a lane keeps 32 bits of address however far the loop goes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
__device__ __forceinline__ uint4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t add) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, add, 0));
}

// LDS reads that are complete on return.  One asm block each: the regions are
// filled by direct loads that the caller has waited for, and for a plain read
// the compiler waits for every one still in flight.
//
// The two 16-byte chunks of two (one) row blocks, at a and a ^ 64 plus 2048 a block ...
template <int N>
__device__ __forceinline__ void read_rows(uint32_t a, v4i (&lo)[2], v4i (&hi)[2]) {
  const uint32_t b = a ^ 64u;
  if constexpr (N == 2)
    asm volatile(
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %4 offset:2048\n\t"
        "ds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1])
        : "v"(a), "v"(b)
        : "memory");
  else
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0])
                 : "v"(a), "v"(b)
                 : "memory");
}
// ... and with them the rows' scale bytes, at c and c + 4 plus 320 (16 pitches) a block
template <int N>
__device__ __forceinline__ void read_rows_scales(uint32_t a, uint32_t c, v4i (&lo)[2], v4i (&hi)[2], uint32_t (&s0)[2],
                                                 uint32_t (&s1)[2]) {
  const uint32_t b = a ^ 64u;
  if constexpr (N == 2)
    asm volatile(
        "ds_read_u8 %4, %10\n\tds_read_u8 %5, %10 offset:4\n\tds_read_u8 %6, %10 offset:320\n\t"
        "ds_read_u8 %7, %10 offset:324\n\t"
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %8 offset:2048\n\t"
        "ds_read_b128 %3, %9 offset:2048\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(s0[0]), "=&v"(s1[0]), "=&v"(s0[1]), "=&v"(s1[1])
        : "v"(a), "v"(b), "v"(c)
        : "memory");
  else
    asm volatile(
        "ds_read_u8 %2, %6\n\tds_read_u8 %3, %6 offset:4\n\tds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(s0[0]), "=&v"(s1[0])
        : "v"(a), "v"(b), "v"(c)
        : "memory");
}
// The scale bytes of CF weight rows at a[f], and at a[f] + 4.
template <int CF>
__device__ __forceinline__ void read_scales(const uint32_t (&a)[CF], uint32_t add, uint32_t (&s0)[CF], uint32_t (&s1)[CF]) {
  if constexpr (CF == 4)
    asm volatile(
        "ds_read_u8 %0, %8\n\tds_read_u8 %1, %9\n\tds_read_u8 %2, %10\n\tds_read_u8 %3, %11\n\t"
        "ds_read_u8 %4, %8 offset:4\n\tds_read_u8 %5, %9 offset:4\n\tds_read_u8 %6, %10 offset:4\n\t"
        "ds_read_u8 %7, %11 offset:4\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(s0[0]), "=&v"(s0[1]), "=&v"(s0[2]), "=&v"(s0[3]), "=&v"(s1[0]), "=&v"(s1[1]), "=&v"(s1[2]), "=&v"(s1[3])
        : "v"(a[0] + add), "v"(a[1] + add), "v"(a[2] + add), "v"(a[3] + add)
        : "memory");
  else
    asm volatile("ds_read_u8 %0, %2\n\tds_read_u8 %1, %2 offset:4\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(s0[0]), "=&v"(s1[0])
                 : "v"(a[0] + add)
                 : "memory");
}

// A group of m rows: as few tiles as hold them, evenly filled with blocks of 16.
__device__ __forceinline__ int row_tiles(int m) { return (m + kRows - 1) / kRows; }
__device__ __forceinline__ int tile_frags(int m, int nb) { return ((m + 15) / 16 + nb - 1) / nb; }

struct Tile {
  int64_t row0, col0;
  int g, rows;
};

// The kernel's LDS.
template <bool A8>
struct Lds {
  uint8_t x[kStages][kStageBytes];
  uint8_t ws[2][64 * kWaves * kPitch];           // weight scales of two windows, 64 columns a wave
  uint8_t xs[2][A8 ? 16 : kRows * kPitch];       // 4-bit rows: their scales
  float ls[A8 ? kRows : 4];                      // e4m3 rows: their scales
  int4 desc[kDesc];
};

// One tile, MI row blocks of 16: each wave all its rows by 16 CF columns.
//
// Per stage (128 bytes of a row: 128 e4m3 or 256 4-bit elements) the rows go
// to LDS by direct loads, two stages ahead, and are read by all four waves.
// A wave's weights are nobody else's, so they go straight to its registers,
// NB - 1 stages ahead.  Scale bytes come to LDS a window of 16 blocks at a
// time (a block's byte alone would fetch a whole cache line).
// Weight row of fragment f at lane n = l%16: column 4 CF (n / 4) + 4 f + n % 4
// of the wave's, so that output lane l holds 4 CF consecutive columns.
template <bool A8, bool OUT_BF16, int CF, int MI>
__device__ __forceinline__ void run_tile(const Mx4Args& p, Lds<A8>& sm, const Tile& t) {
  constexpr int PPS = A8 ? 1 : 2;                // 128-element pieces a stage
  constexpr int NB = CF == 4 ? 2 : 3;            // weight register buffers
  constexpr int SPW = 4 / PPS;                   // stages a scale window
  constexpr int ROWS = 16 * MI;
  constexpr int XFULL = MI / 2, XHALF = MI & 1;  // a wave's direct loads of rows a stage: 8 rows each, and 4
  constexpr int ND = XFULL + XHALF, NWL = CF * PPS;
  const int tid = opaque(threadIdx.x);
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l15 = lane & 15, grp = lane >> 4;
  const int kb = static_cast<int>(p.K / 32);
  const int xbytes = static_cast<int>(A8 ? p.K : p.K / 2), wbytes = static_cast<int>(p.K / 2);
  const int NS = (xbytes + 127) / 128;
  const int nwin = (kb + 15) / 16;

  // direct loads of rows: lane l fills slot l%8 of row R + l/8; rows past the tile's repeat its last
  const __amdgpu_buffer_rsrc_t xbuf = buffer(p.lhs + t.row0 * p.ldl, static_cast<uint32_t>((t.rows - 1) * p.ldl + xbytes));
  uint32_t xoff[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const int r = 4 * MI * wave + 8 * i + (lane >> 3);
    xoff[i] = static_cast<uint32_t>(min(r, t.rows - 1)) * static_cast<uint32_t>(p.ldl) + 16 * ((lane & 7) ^ swz(r));
  }
  auto load_rows = [&](int s, auto end_c) {
    uint8_t* dst = sm.x[s % kStages] + 4 * MI * wave * 128;
    if (!decltype(end_c)::value || 128 * s + 128 <= xbytes) {
#pragma unroll
      for (int i = 0; i < ND; ++i)
        if (i < XFULL || lane < 32)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_void*)(dst + 1024 * i), 16, xoff[i], 128 * s, 0, 0);
    } else {                                     // chunks past the row: its last one (their weights are zero)
      const int ln = opaque(lane);
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        const int at = 128 * s + 16 * ((ln & 7) ^ swz(4 * MI * wave + 8 * i + (ln >> 3)));
        if (i < XFULL || lane < 32)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_void*)(dst + 1024 * i), 16,
                                                   xoff[i] + 128 * s - max(at - (xbytes - 16), 0), 0, 0, 0);
      }
    }
  };

  // weights into registers
  const int64_t colw = t.col0 + 16 * CF * wave;  // the wave's first column
  const int last_col = static_cast<int>(max(min(p.N - 1 - colw, static_cast<int64_t>(16 * CF - 1)), static_cast<int64_t>(0)));
  const int colc = static_cast<int>(min(colw, p.N - 1));                     // a wave past the last column repeats it
  const __amdgpu_buffer_rsrc_t wbuf =
      buffer(p.rhs + (static_cast<int64_t>(t.g) * p.N + colc) * wbytes, static_cast<uint32_t>(last_col + 1) * wbytes);
  uint32_t woff[CF], wsa[CF];
  const uint8_t* wsbase = p.rs + static_cast<int64_t>(t.g) * p.N * kb;
#pragma unroll
  for (int f = 0; f < CF; ++f) {
    const int r = 4 * CF * (l15 >> 2) + 4 * f + (l15 & 3), rc = min(r, last_col);
    woff[f] = static_cast<uint32_t>(rc) * static_cast<uint32_t>(wbytes) + 16 * grp;
    // this lane's scale byte of the row, at block 4 piece + l/16
    wsa[f] = lds_addr(sm.ws[0]) + (wave * 64 + r) * kPitch + ((static_cast<uint32_t>(colc + rc) * kb) & 3) + grp;
  }
  uint4 w[NB][CF][PPS];
  auto load_weights = [&](int s, uint4 (&b)[CF][PPS], auto end_c) {
#pragma unroll
    for (int u = 0; u < PPS; ++u) {
      const int at = 64 * (PPS * s + u);
      if (!decltype(end_c)::value || at + 64 <= wbytes) {
#pragma unroll
        for (int f = 0; f < CF; ++f) b[f][u] = buffer_load16(wbuf, woff[f], at);
      } else {                                   // pieces past the row: its last one
        const int back = max(at + 16 * grp - (wbytes - 16), 0);
#pragma unroll
        for (int f = 0; f < CF; ++f) b[f][u] = buffer_load16(wbuf, woff[f] + at - back, 0);
      }
    }
  };

  // Scale windows: row r's 16 bytes from byte r * stride + 16 w, fetched as the five dwords around them;
  // five lanes a row.  Dwords past the array's last are that one (their bytes are not used).
  auto load_scales = [&](int win) {
    const int ln = opaque(lane);
    const uint32_t ws_last = static_cast<uint32_t>(p.N * kb / 4 - 1);
    uint8_t* dst = sm.ws[win & 1] + wave * 64 * kPitch;
#pragma unroll
    for (int i = 0; i < (80 * CF + 63) / 64; ++i) {
      const int idx = 64 * i + ln, r = idx / 5, d = idx - 5 * r;
      const uint32_t row = colc + min(r, last_col);
      const uint32_t dw = min((row * kb + 16 * win) / 4 + d, ws_last);
      if (r < 16 * CF) __builtin_amdgcn_global_load_lds(wsbase + 4 * dw, (lds_void*)(dst + 256 * i), 4, 0, 0);
    }
    if constexpr (!A8) {
      uint8_t* xd = sm.xs[win & 1] + wave * 4 * MI * kPitch;
      const uint8_t* base = static_cast<const uint8_t*>(p.ls) + t.row0 * p.lds;
      const int64_t end = (p.M - t.row0 - 1) * p.lds + ((kb + 3) & ~3) - 4;      // last dword that holds scales
#pragma unroll
      for (int i = 0; i < (20 * MI + 63) / 64; ++i) {
        const int idx = 64 * i + ln, r = idx / 5, d = idx - 5 * r;
        const int row = min(4 * MI * wave + r, t.rows - 1);
        const int64_t off = min(static_cast<int64_t>(row) * p.lds + 16 * win + 4 * d, end);
        if (r < 4 * MI) __builtin_amdgcn_global_load_lds(base + off, (lds_void*)(xd + 256 * i), 4, 0, 0);
      }
    }
  };

  v4f acc[MI][CF];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int f = 0; f < CF; ++f) acc[i][f] = v4f{0.f, 0.f, 0.f, 0.f};

  step_barrier();                                // the last tile's readers are done
  if constexpr (A8) {
    if (tid < ROWS)
      __builtin_amdgcn_global_load_lds(static_cast<const float*>(p.ls) + (p.ls_per_row ? t.row0 + min(tid, t.rows - 1) : 0),
                                       (lds_void*)(sm.ls + 64 * wave), 4, 0, 0);
  }
  load_scales(0);
  order();
#pragma unroll
  for (int u = 0; u < NB - 1; ++u)
    if (u < NS) load_weights(u, w[u], std::true_type());
  order();
  load_rows(0, std::true_type());
  order();
  if (NS > 1) {
    load_rows(1, std::true_type());
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(ND));
  } else {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  }

  const uint32_t xa0 = lds_addr(sm.x[0]) + l15 * 128 + 16 * (grp ^ swz(l15));
  const uint32_t xsa0 = lds_addr(sm.xs[0]) + l15 * kPitch + grp;
  // Stage s, its weights in buffer u.  END: the last stages, where what would be loaded may not exist and
  // the last blocks may lie past K; before them every load is whole and the counts are constants.
  auto stage = [&](int s, auto u_c, auto end_c) {
    constexpr int u = decltype(u_c)::value;
    constexpr bool END = decltype(end_c)::value;
    step_barrier();                              // every wave's rows of stage s are there; stage s - 1 is read
    if (s % SPW == 0 && s / SPW + 1 < nwin) load_scales(s / SPW + 1);
    order();
    if (!END || s + NB - 1 < NS) load_weights(s + NB - 1, w[(u + NB - 1) % NB], end_c);
    order();
    if (!END || s + 2 < NS) load_rows(s + 2, end_c);
    order();
    const int win = (s / SPW) & 1;
    uint32_t ws0[CF], ws1[CF];
    read_scales<CF>(wsa, 4 * PPS * (s % SPW) + win * static_cast<int>(sizeof(sm.ws[0])), ws0, ws1);
    if (END && s + 1 == NS) {                    // blocks past K: zero weights with a plain scale
#pragma unroll
      for (int q = 0; q < PPS; ++q) {
        const bool past = 4 * (PPS * s + q) + grp >= kb;
#pragma unroll
        for (int f = 0; f < CF; ++f) {
          w[u][f][q].x = past ? 0 : w[u][f][q].x;
          w[u][f][q].y = past ? 0 : w[u][f][q].y;
          w[u][f][q].z = past ? 0 : w[u][f][q].z;
          w[u][f][q].w = past ? 0 : w[u][f][q].w;
          if (q) ws1[f] = past ? 127 : ws1[f];
          else ws0[f] = past ? 127 : ws0[f];
        }
      }
    }
    const uint32_t xa = xa0 + (s % kStages) * kStageBytes;
    const uint32_t xsa = xsa0 + 8 * (s % SPW) + win * static_cast<int>(sizeof(sm.xs[0]));
#pragma unroll
    for (int i0 = 0; i0 < MI; i0 += 2) {
      constexpr int N = MI == 1 ? 1 : 2;
      static_assert(MI % N == 0, "row blocks are read in pairs");
      v4i lo[2], hi[2];
      uint32_t xs0[2] = {127, 127}, xs1[2] = {127, 127};
      if constexpr (A8)
        read_rows<N>(xa + 2048 * i0, lo, hi);
      else
        read_rows_scales<N>(xa + 2048 * i0, xsa + 16 * kPitch * i0, lo, hi, xs0, xs1);
#pragma unroll
      for (int q = 0; q < N; ++q) {
#pragma unroll
        for (int f = 0; f < CF; ++f) {
          v4f& c = acc[i0 + q][f];
          if constexpr (A8) {
            const v8i xv = {lo[q][0], lo[q][1], lo[q][2], lo[q][3], hi[q][0], hi[q][1], hi[q][2], hi[q][3]};
            c = mfma_mx4<true>(frag16(w[u][f][0]), ws0[f], xv, 127, c);
          } else {
            const v8i x0 = {lo[q][0], lo[q][1], lo[q][2], lo[q][3], 0, 0, 0, 0};
            const v8i x1 = {hi[q][0], hi[q][1], hi[q][2], hi[q][3], 0, 0, 0, 0};
            c = mfma_mx4<false>(frag16(w[u][f][0]), ws0[f], x0, xs0[q], c);
            c = mfma_mx4<false>(frag16(w[u][f][PPS - 1]), ws1[f], x1, xs1[q], c);
          }
        }
      }
      // reads the pair's sums, so that its products are issued here: left free, the compiler moves them behind
      // the next reads, and holds every block's rows until then
#pragma unroll
      for (int q = 0; q < N; ++q) {
        if constexpr (CF == 4)
          asm volatile("" : "+v"(acc[i0 + q][0]), "+v"(acc[i0 + q][1]), "+v"(acc[i0 + q][2]), "+v"(acc[i0 + q][3]));
        else
          asm volatile("" ::"v"(acc[i0 + q][0]));
      }
    }
    // this wave's rows of stage s + 1 have landed when only what this stage issued after them is outstanding:
    // its weights and the rows of stage s + 2 (loads complete in order; the scale window was issued before both)
    if (!END || s + 2 < NS)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(ND + NWL));
    else
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  };
  using std::integral_constant;
  int s0 = 0;
#pragma clang loop unroll(disable)
  for (; s0 + NB + 2 <= NS; s0 += NB) {          // the furthest load is of stage s0 + NB + 1, which may be partial
    stage(s0, integral_constant<int, 0>(), std::false_type());
    stage(s0 + 1, integral_constant<int, 1>(), std::false_type());
    if constexpr (NB == 3) stage(s0 + 2, integral_constant<int, 2>(), std::false_type());
  }
#pragma clang loop unroll(disable)
  for (; s0 < NS; s0 += NB) {
    stage(s0, integral_constant<int, 0>(), std::true_type());
    if (s0 + 1 < NS) stage(s0 + 1, integral_constant<int, 1>(), std::true_type());
    if constexpr (NB == 3)
      if (s0 + 2 < NS) stage(s0 + 2, integral_constant<int, 2>(), std::true_type());
  }

  // output: this lane's row of every block, 4 CF consecutive columns
  const int64_t c = colw + 4 * CF * grp;
  if (c < p.N) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = 16 * i + l15;
      if (r >= t.rows) continue;
      const float lsr = A8 ? sm.ls[r] : 1.0f;
      const int64_t at = (t.row0 + r) * p.N + c;
      if (OUT_BF16) {
        uint32_t o[2 * CF];
#pragma unroll
        for (int f = 0; f < CF; ++f)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            o[2 * f + q] = f32_to_bf16(acc[i][f][2 * q] * lsr) |
                           (static_cast<uint32_t>(f32_to_bf16(acc[i][f][2 * q + 1] * lsr)) << 16);
        uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at);
        if constexpr (CF == 4) {
          reinterpret_cast<uint4*>(d)[0] = make_uint4(o[0], o[1], o[2], o[3]);
          reinterpret_cast<uint4*>(d)[1] = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
          *reinterpret_cast<uint2*>(d) = make_uint2(o[0], o[1]);
        }
      } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
        for (int f = 0; f < CF; ++f)
          d[f] = make_float4(acc[i][f][0] * lsr, acc[i][f][1] * lsr, acc[i][f][2] * lsr, acc[i][f][3] * lsr);
      }
    }
  }
}

// Persistent workgroups of four waves, two a CU.  A tile is up to 128 rows of
// one group by 64 CF columns; the tile range is split over the XCDs, row
// tiles fastest, so that a group's weights are fetched once and shared in L2.
template <bool A8, bool OUT_BF16, int CF>
__global__ __launch_bounds__(kThreads, 2) void gmm_mx4_kernel(const Mx4Args p) {
  __shared__ __attribute__((aligned(1024))) Lds<A8> sm;
  constexpr int BN = 64 * CF;
  const int NT = static_cast<int>((p.N + BN - 1) / BN);
  // the group table lives in the stages while tiles are decoded, up to kDesc at a time
  struct Table {
    int rows_off[kMaxLocal + 1], tiles_off[kMaxLocal + 1], tmp[kMaxLocal];
  };
  static_assert(sizeof(Table) <= sizeof(sm.x), "the group table fits the stages");
  Table& gt = *reinterpret_cast<Table*>(&sm.x[0][0]);
  int first = 0, last = 0, step = 1, n_rows = 0;
#pragma clang loop unroll(disable)
  for (int base = 0;; base += kDesc) {
    const int tid = opaque(threadIdx.x);
    __syncthreads();
    for (int g = tid; g < p.El; g += kThreads) {
      int m = p.group_sizes[p.g0 + g];
      if (m < 0) {
        if (blockIdx.x == 0) raise_error(p.err, MOE_DEVERR_GROUP_SIZE);
        m = 0;
      }
      gt.tmp[g] = m;
    }
    __syncthreads();
    const bool over = wave0_scan_sat(gt.tmp, gt.rows_off, p.El, p.M);
    if (over && tid == 0 && blockIdx.x == 0) raise_error(p.err, MOE_DEVERR_ROWS);
    __syncthreads();
    for (int g = tid; g < p.El; g += kThreads) gt.tmp[g] = row_tiles(gt.rows_off[g + 1] - gt.rows_off[g]) * NT;
    __syncthreads();
    wave0_scan(gt.tmp, gt.tiles_off, p.El);
    __syncthreads();
    xcd_share(gt.tiles_off[p.El], first, last, step);
    n_rows = gt.rows_off[p.El];
    const int left = first < last ? (last - first + step - 1) / step - base : 0;       // this workgroup's tiles
    if (tid < min(left, kDesc)) {
      const int t = first + (base + tid) * step;
      const int g = find_group(gt, p.El, t);
      const int m = gt.rows_off[g + 1] - gt.rows_off[g], nb = row_tiles(m), fr = tile_frags(m, nb);
      const int local = t - gt.tiles_off[g], ct = local / nb, rt = local - ct * nb;
      // (even filling may leave a last tile without rows)
      sm.desc[tid] = make_int4(gt.rows_off[g] + 16 * fr * rt, ct, g, min(16 * fr, m - 16 * fr * rt));
    }
    __syncthreads();
    for (int i = 0; i < min(left, kDesc); ++i) {
      const int4 d = sm.desc[i];
      Tile t;
      t.row0 = __builtin_amdgcn_readfirstlane(d.x);
      t.col0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(d.y)) * BN;
      t.g = __builtin_amdgcn_readfirstlane(d.z);
      t.rows = __builtin_amdgcn_readfirstlane(d.w);
      if (t.rows <= 0) continue;
      if (t.rows <= 16) run_tile<A8, OUT_BF16, CF, 1>(p, sm, t);
      else if (t.rows <= 32) run_tile<A8, OUT_BF16, CF, 2>(p, sm, t);
      else if (t.rows <= 64) run_tile<A8, OUT_BF16, CF, 4>(p, sm, t);
      else if (t.rows <= 96) run_tile<A8, OUT_BF16, CF, 6>(p, sm, t);
      else run_tile<A8, OUT_BF16, CF, 8>(p, sm, t);
    }
    if (left <= kDesc) break;
  }
  // rows past the last group's are zero
  const int64_t bytes = (p.M - n_rows) * p.N * (OUT_BF16 ? 2 : 4);
  uint8_t* z = static_cast<uint8_t*>(p.out) + n_rows * p.N * (OUT_BF16 ? 2 : 4);
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + opaque(threadIdx.x)) * 16; i < bytes;
       i += static_cast<int64_t>(gridDim.x) * kThreads * 16)
    *reinterpret_cast<uint4*>(z + i) = make_uint4(0, 0, 0, 0);
}

// Scale rows that are not dword aligned, copied to rows that are.
__global__ __launch_bounds__(256) void align_scales_kernel(const uint8_t* __restrict__ s, int64_t lds, int64_t M, int kb,
                                                           uint8_t* __restrict__ out, int64_t ldo) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < M * kb; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / kb, b = i - r * kb;
    out[r * ldo + b] = s[r * lds + b];
  }
}

template <bool A8, bool OUT_BF16>
hipError_t launch(const Mx4Args& p, hipStream_t st) {
  // 256-column tiles when they fill the GPU's workgroups, 64-column ones otherwise
  const int64_t groups = p.El < p.M ? p.El : p.M;
  const int64_t row_t = groups + p.M / kRows;
  const int64_t slots = 2 * num_cus();
  const bool wide = row_t * moe_cdiv(p.N, 256) >= slots;
  const int64_t most = (moe_cdiv(p.M, kRows) + groups) * moe_cdiv(p.N, wide ? 256 : 64);
  const int64_t grid = most < 8 ? 8 : most < slots ? most : slots;       // each XCD's part has its own workgroups
  if (wide)
    gmm_mx4_kernel<A8, OUT_BF16, 4><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
  else
    gmm_mx4_kernel<A8, OUT_BF16, 1><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

// The error word, and room for dword-aligned scale rows of a 4-bit lhs.
size_t gmm_mx4_ws_bytes(int64_t M, int64_t K) {
  return static_cast<size_t>(tile::kHdr) + static_cast<size_t>((M * ((K / 32 + 3) / 4 * 4) + 255) / 256 * 256);
}

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
  // row offsets inside a tile, and a group's weights' scale bytes, are 32-bit
  if (M > INT32_MAX - 1 || K > (1 << 22) || ldl > (1 << 23) || N > INT32_MAX || N * (K / 32) > INT32_MAX) return MOE_ERR_SHAPE;
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
      reinterpret_cast<uintptr_t>(rhs_scale) % 16 || reinterpret_cast<uintptr_t>(out) % 16)
    return MOE_ERR_SHAPE;
  if (!ws || ws_bytes < moe::gmm_mx4_ws_bytes(M, K)) return MOE_ERR_WORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  moe::Mx4Args p{lhs, ldl, lhs_scale, lds, lhs_scale_mode == MOE_SCALE_ROW_DYNAMIC ? 1 : 0, rhs, rhs_scale,
                 group_sizes, group_offset, num_local_experts, M, K, N, out, static_cast<int32_t*>(ws)};
  if (!a8 && num_local_experts > 0 && (lds % 4 || reinterpret_cast<uintptr_t>(lhs_scale) % 4)) {
    const int kb = static_cast<int>(K / 32);
    uint8_t* rows = static_cast<uint8_t*>(ws) + moe::tile::kHdr;
    const int64_t ldo = (kb + 3) / 4 * 4, blocks = moe_cdiv(M * kb, 256);
    moe::align_scales_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, st>>>(
        static_cast<const uint8_t*>(lhs_scale), lds, M, kb, rows, ldo);
    MOE_CHECK_LAUNCH();
    p.ls = rows;
    p.lds = ldo;
  }
  hipError_t e;
  if (a8)
    e = out_dtype == MOE_BF16 ? moe::launch<true, true>(p, st) : moe::launch<true, false>(p, st);
  else
    e = out_dtype == MOE_BF16 ? moe::launch<false, true>(p, st) : moe::launch<false, false>(p, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
