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
//
// Three kernels, all persistent, by format and size:
//   4-bit rows, 256 x 256 tiles (run_wide): 8192 rows of 7168 by 32 groups of
//     4096 columns 218 us in the trace, 2.2 PFLOP/s (as calls 229; with 128
//     rows a tile 238, as run_tile 259).  Loads bound it: without its products
//     and LDS reads a call took 207 us.
//   e4m3 rows, 128 x 256 tiles (run_tile, 4 column fragments a wave): 32768
//     rows of 2048 by 64 groups of 1536 columns 122 us, 1.68 PFLOP/s (as calls
//     132 then; as 256 x 256 tiles with the weights through LDS 142).
//   fewer tiles than workgroups: 64-column tiles (run_tile, one column
//     fragment a wave): 512 ragged rows of 2080 by 1040 columns 13.5 us (as
//     calls 15; with 256-column tiles 30); the two above would take 352 and 200.
// Weights kept out of the caches (they are read by two row tiles) cost the
// first case 27 us.
#include <type_traits>

#include "mx4_common.hpp"
#include "stage_common.hpp"

namespace moe {
namespace {
using namespace tile;
using namespace stage;
using mx4::quad_exchange;

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
  int tile_rows;               // rows a tile holds at most
};

constexpr int kThreads = 256, kWaves = 4;
constexpr int kRows = 128;                       // rows a tile holds at most
constexpr int kStages = 3;
constexpr int kPitch = 20;                       // LDS bytes a row of one scale window: 16 blocks, at any alignment
constexpr int kDesc = 64;                        // tiles decoded at a time

// Slot of 16-byte chunk c of staged row r: c ^ swz(r).  Eight consecutive rows
// use eight slots, so a fragment read (16 rows, served 8 lanes at a time) is
// free of bank conflicts.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// LDS reads that are complete on return.  One asm block each: the regions are
// filled by direct loads that the caller has waited for, and for a plain read
// the compiler waits for every one still in flight.
//
// e4m3 rows: the two 16-byte chunks of two (one) row blocks, at a and a ^ 64 plus 2048 a block
template <int N>
__device__ __forceinline__ void read_rows8(uint32_t a, v4i (&lo)[2], v4i (&hi)[2]) {
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
// 4-bit rows: the chunk of four (two, one) row blocks, and their scale byte at c plus 320 (16 pitches) a block
template <int N>
__device__ __forceinline__ void read_rows4(uint32_t a, uint32_t c, v4i (&x)[4], uint32_t (&s)[4]) {
  if constexpr (N == 4)
    asm volatile(
        "ds_read_u8 %4, %9\n\tds_read_u8 %5, %9 offset:320\n\tds_read_u8 %6, %9 offset:640\n\t"
        "ds_read_u8 %7, %9 offset:960\n\tds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\t"
        "ds_read_b128 %2, %8 offset:4096\n\tds_read_b128 %3, %8 offset:6144\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2]), "=&v"(s[3])
        : "v"(a), "v"(c)
        : "memory");
  else if constexpr (N == 2)
    asm volatile(
        "ds_read_u8 %2, %5\n\tds_read_u8 %3, %5 offset:320\n\tds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(s[0]), "=&v"(s[1])
        : "v"(a), "v"(c)
        : "memory");
  else
    asm volatile("ds_read_u8 %1, %3\n\tds_read_b128 %0, %2\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(x[0]), "=&v"(s[0])
                 : "v"(a), "v"(c)
                 : "memory");
}
// The scale bytes of CF weight rows, four rows (80 bytes) apart.
template <int CF>
__device__ __forceinline__ void read_scales(uint32_t a, uint32_t (&s)[CF]) {
  if constexpr (CF == 4)
    asm volatile(
        "ds_read_u8 %0, %4\n\tds_read_u8 %1, %4 offset:80\n\tds_read_u8 %2, %4 offset:160\n\t"
        "ds_read_u8 %3, %4 offset:240\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2]), "=&v"(s[3])
        : "v"(a)
        : "memory");
  else if constexpr (CF == 3)
    asm volatile(
        "ds_read_u8 %0, %3\n\tds_read_u8 %1, %3 offset:80\n\tds_read_u8 %2, %3 offset:160\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2])
        : "v"(a)
        : "memory");
  else
    asm volatile("ds_read_u8 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(s[0]) : "v"(a) : "memory");
}

struct Tile {
  int64_t row0, col0;
  int g, rows;
};

// The kernel's LDS.
template <bool A8>
struct Lds {
  uint8_t x[kStages][kRows * 128];
  uint8_t ws[2][64 * kWaves * kPitch];           // weight scales of two windows, 64 columns a wave
  uint8_t xs[2][A8 ? 16 : kRows * kPitch];       // 4-bit rows: their scales
  float ls[A8 ? kRows : 4];                      // e4m3 rows: their scales
  int4 desc[kDesc];
};

// Reads a row block's sums, so that its products are issued here: left free,
// the compiler moves them behind the next reads, and holds every block's rows
// until then.
template <int CF>
__device__ __forceinline__ void pin(const v4f (&c)[CF]) {
  if constexpr (CF == 4)
    asm volatile("" ::"v"(c[0]), "v"(c[1]), "v"(c[2]), "v"(c[3]));
  else if constexpr (CF == 3)
    asm volatile("" ::"v"(c[0]), "v"(c[1]), "v"(c[2]));
  else
    asm volatile("" ::"v"(c[0]));
}

// This lane's row r0 + 16 i + l%16 of every block, 4 CF consecutive columns from c.
template <bool A8, bool OUT_BF16, int CF, int MI>
__device__ __forceinline__ void store_tile(const Mx4Args& p, const Tile& t, const v4f (&acc)[MI][CF], const float* ls, int r0,
                                           int64_t c, int l15) {
  if (c >= p.N) return;                          // N is a multiple of 16: all of the lane's columns exist, or none
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = r0 + 16 * i + l15;
    if (r >= t.rows) continue;
    const float lsr = A8 ? ls[r] : 1.0f;
    const int64_t at = (t.row0 + r) * p.N + c;
    if (OUT_BF16) {
      uint32_t o[2 * CF];
#pragma unroll
      for (int f = 0; f < CF; ++f)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          o[2 * f + q] = f32_to_bf16(acc[i][f][2 * q] * lsr) |
                         (static_cast<uint32_t>(f32_to_bf16(acc[i][f][2 * q + 1] * lsr)) << 16);
      uint16_t* d = static_cast<uint16_t*>(p.out) + at;
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

// Pieces q0 .. q0 + N - 1 (those below `end`).
template <int N, int U = 0, class F, class E>
__device__ __forceinline__ void pieces(const F& piece, int q0, E end_c, int end = 0) {
  if constexpr (U < N) {
    if (!E::value || q0 + U < end) piece(q0 + U, std::integral_constant<int, U>(), end_c);
    pieces<N, U + 1>(piece, q0, end_c, end);
  }
}

// 0 .. MI - 1 in blocks of N, what is left in blocks of half that.
template <int N, int MI, int I0 = 0, class F>
__device__ __forceinline__ void in_blocks(const F& blocks) {
  if constexpr (I0 < MI) {
    if constexpr (I0 + N <= MI) {
      blocks(std::integral_constant<int, I0>(), std::integral_constant<int, N>());
      in_blocks<N, MI, I0 + N>(blocks);
    } else {
      in_blocks<N / 2, MI, I0>(blocks);
    }
  }
}

// One tile, MI row blocks of 16: each wave all its rows by 16 CF columns.
//
// Per stage (128 bytes of a row: one piece of 128 e4m3 elements or two of 128
// 4-bit ones) the rows go to LDS by direct loads, two stages ahead, and are
// read by all four waves.  A wave's weights are nobody else's, so they go
// straight to its registers, a set of four fragments ahead (four of one piece,
// or one of four pieces), each load 64 bytes of 16 rows and the lanes exchanged
// (quad_exchange): as plain fragment loads, 16 bytes of 64 rows, the address
// unit bounds the kernel.  Scale bytes come to LDS a window of 16 blocks at a
// time (a block's byte alone would fetch a whole cache line).
// Weight row of fragment f at lane n = l%16: column 4 CF (n / 4) + 4 f + n % 4
// of the wave's, so that output lane l holds 4 CF consecutive columns.
template <bool A8, bool OUT_BF16, int CF, int MI>
__device__ __forceinline__ void run_tile(const Mx4Args& p, Lds<A8>& sm, const Tile& t) {
  constexpr int PPS = A8 ? 1 : 2;                // 128-element pieces a stage
  constexpr int SPW = 4 / PPS;                   // stages a scale window
  constexpr int ROWS = 16 * MI;
  constexpr int XFULL = MI / 2, XHALF = MI & 1;  // a wave's direct loads of rows a stage: 8 rows each, and 4
  // weights are loaded by sets of four fragments (quad_exchange): the four of a piece, or four pieces of the one
  constexpr int UNIT = CF == 4 ? 1 : 4;          // pieces a set
  constexpr int NB = 2;                          // register buffers, a set each: one set ahead
  constexpr int UNROLL = NB * UNIT;
  constexpr int ND = XFULL + XHALF, NWL = CF == 4 ? 4 * PPS : 4;             // a wave's loads: of rows a stage, of weights
  const int tid = opaque(threadIdx.x);
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l15 = lane & 15, grp = lane >> 4;
  const int kb = static_cast<int>(p.K / 32);
  const int xbytes = static_cast<int>(A8 ? p.K : p.K / 2), wbytes = static_cast<int>(p.K / 2);
  const int NP = (kb + 3) / 4;                   // pieces
  const int NS = (NP + PPS - 1) / PPS;           // stages
  const int NU = (NS * PPS + UNIT - 1) / UNIT;   // sets
  const int nwin = (kb + 15) / 16;

  // Direct loads of rows: lane l fills slot l%8 of row R + l/8.  Rows past the tile's last lie outside the
  // buffer (zeros).  The slot's chunk alternates with every 8 rows: two lane offsets.
  const uint32_t ldl = static_cast<uint32_t>(p.ldl);
  const __amdgpu_buffer_rsrc_t xbuf = buffer(p.lhs + t.row0 * p.ldl, (t.rows - 1) * ldl + xbytes);
  const int r0 = 4 * MI * wave + (lane >> 3);
  const uint32_t xoff = r0 * ldl;
  const int xc = 16 * ((lane & 7) ^ swz(r0));
  auto load_rows = [&](int s, auto end_c) {
    uint8_t* dst = sm.x[s % kStages] + 4 * MI * wave * 128;
    // chunks past the row: its last one (their weights are zero)
    const bool part = decltype(end_c)::value && 128 * s + 128 > xbytes;
    const int lim = xbytes - 16 - 128 * s;
    const uint32_t o0 = xoff + (part ? min(static_cast<int>(xc), lim) : xc);
    const uint32_t o1 = xoff + (part ? min(static_cast<int>(xc ^ 16), lim) : xc ^ 16);
#pragma unroll
    for (int i = 0; i < ND; ++i)
      if (i < XFULL || lane < 32)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_void*)(dst + 1024 * i), 16, i & 1 ? o1 : o0, 128 * s + 8 * i * ldl, 0, 0);
  };

  // weights into registers; columns past N lie outside the buffer (zeros, and never stored)
  const int64_t colw = t.col0 + 16 * CF * wave;  // the wave's first column
  const int last_col = static_cast<int>(max(min(p.N - 1 - colw, static_cast<int64_t>(16 * CF - 1)), static_cast<int64_t>(0)));
  const int colc = static_cast<int>(min(colw, p.N - 1));                     // a wave past the last column repeats it
  const __amdgpu_buffer_rsrc_t wbuf =
      buffer(p.rhs + (static_cast<int64_t>(t.g) * p.N + colc) * wbytes, static_cast<uint32_t>(last_col + 1) * wbytes);
  const int wr = 4 * CF * (l15 >> 2) + (l15 & 3);                            // weight row of fragment 0; 4 f more for f
  // load i, lane 16 h + 4 m + c: chunk c of weight row 4 m + i of fragment h (of the one fragment, piece h)
  const int wl = CF == 4 ? 16 * ((lane >> 2) & 3) + 4 * (lane >> 4) : 4 * ((lane >> 2) & 3);
  const uint32_t wk = 16 * (lane & 3) + (CF == 4 ? 0 : 64 * (lane >> 4));
  const uint32_t woff = static_cast<uint32_t>(wl) * wbytes + wk;
  uint4 w[NB][4];
  auto load_weights = [&](int un, uint4 (&b)[4], auto end_c) {
    const int at = 64 * UNIT * un;
    uint32_t o = woff;
    if (decltype(end_c)::value) o -= max(at + static_cast<int>(wk) - (wbytes - 16), 0);     // chunks past the row: its last one
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = buffer_load16(wbuf, o, at + i * wbytes);
  };

  // Scale windows: row r's 16 bytes from byte r * stride + 16 w, fetched as the five dwords around them;
  // five lanes a row.  Dwords past the array's last are that one (their bytes are not used).
  const uint8_t* wsbase = p.rs + static_cast<int64_t>(t.g) * p.N * kb;
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
    if (u < NU) load_weights(u, w[u], std::true_type());
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
  // this lane's scale byte of weight row wr, at block 4 piece + l/16 (rows 4 f on start at the same byte of a dword)
  const uint32_t wsa0 = lds_addr(sm.ws[0]) + (wave * 64 + wr) * kPitch + ((static_cast<uint32_t>(colc + wr) * kb) & 3) + grp;

  // Piece q = UNROLL n + u, its weights in buffer (u / UNIT) % NB: the first piece of a stage starts it, the last
  // one ends it.  END: the last pieces, where what would be loaded may not exist and the last blocks may lie past K;
  // before them every load is whole and the counts are constants.
  auto piece = [&](int q, auto u_c, auto end_c) {
    constexpr int u = decltype(u_c)::value, h = u % PPS, bu = u / UNIT % NB;
    constexpr bool END = decltype(end_c)::value;
    const int s = q / PPS;
    if (h == 0) {
      step_barrier();                            // every wave's rows of stage s are there; stage s - 1 is read
      if (s % SPW == 0 && s / SPW + 1 < nwin) load_scales(s / SPW + 1);
      order();
    }
    if (u % UNIT == 0) {
      quad_exchange(w[bu], lane);
      __builtin_amdgcn_sched_barrier(0);
      if (!END || q / UNIT + NB - 1 < NU) load_weights(q / UNIT + NB - 1, w[(bu + NB - 1) % NB], end_c);
    }
    order();
    if (h == 0 && (!END || s + 2 < NS)) load_rows(s + 2, end_c);
    order();
    // fragment f of this piece
    auto wf = [&](int f) -> uint4& { return w[bu][CF == 4 ? f : u % 4]; };
    const int win = (q / 4) & 1;
    uint32_t ws[CF];
    read_scales<CF>(wsa0 + 4 * (q % 4) + win * static_cast<int>(sizeof(sm.ws[0])), ws);
    // blocks past K: zero weights, and plain scales for both operands (a 4-bit row's byte there is not its own: it lies
    // between the rows or is the next row's, and a NaN would turn the zeros into NaN)
    const bool past = END && 4 * q + grp >= kb;
    if (END && q >= NP - 1) {
#pragma unroll
      for (int f = 0; f < CF; ++f) {
        wf(f).x = past ? 0 : wf(f).x;
        wf(f).y = past ? 0 : wf(f).y;
        wf(f).z = past ? 0 : wf(f).z;
        wf(f).w = past ? 0 : wf(f).w;
        ws[f] = past ? 127 : ws[f];
      }
    }
    const uint32_t xa = (xa0 ^ (64 * h)) + (s % kStages) * static_cast<int>(sizeof(sm.x[0]));
    const uint32_t xsa = xsa0 + 4 * (q % 4) + win * static_cast<int>(sizeof(sm.xs[0]));
    // row blocks i0 .. i0 + N - 1
    auto blocks = [&](auto i0_c, auto n_c) {
      constexpr int i0 = decltype(i0_c)::value, N = decltype(n_c)::value;
      if constexpr (A8) {
        v4i lo[2], hi[2];
        read_rows8<N>(xa + 2048 * i0, lo, hi);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const v8i x = {lo[j][0], lo[j][1], lo[j][2], lo[j][3], hi[j][0], hi[j][1], hi[j][2], hi[j][3]};
#pragma unroll
          for (int f = 0; f < CF; ++f) acc[i0 + j][f] = mfma_mx4<true>(frag16(wf(f)), ws[f], x, 127, acc[i0 + j][f]);
          pin<CF>(acc[i0 + j]);
        }
      } else {
        v4i x[4];
        uint32_t xs[4];
        read_rows4<N>(xa + 2048 * i0, xsa + 16 * kPitch * i0, x, xs);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (END) xs[j] = past ? 127 : xs[j];
          const v8i xv = {x[j][0], x[j][1], x[j][2], x[j][3], 0, 0, 0, 0};
#pragma unroll
          for (int f = 0; f < CF; ++f) acc[i0 + j][f] = mfma_mx4<false>(frag16(wf(f)), ws[f], xv, xs[j], acc[i0 + j][f]);
          pin<CF>(acc[i0 + j]);
        }
      }
    };
    in_blocks<A8 ? 2 : 4, MI>(blocks);
    // this wave's rows of stage s + 1 have landed when only what was issued after them is outstanding: at least
    // this stage's weights, if it loads any, and the rows of stage s + 2 (loads complete in order)
    if (h == PPS - 1) {
      if (!END || s + 2 < NS)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(ND + (!END && (CF == 4 || (u - h) % UNIT == 0) ? NWL : 0)));
      else
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    }
  };
  int q0 = 0;
  const int whole = static_cast<int>(p.K / 128);           // pieces inside K
  // the furthest loads, of the sets and of the two stages after these pieces, are whole
  constexpr int AHEAD = UNIT * (NB - 1) > 2 * PPS ? UNIT * (NB - 1) : 2 * PPS;
#pragma clang loop unroll(disable)
  for (; q0 + UNROLL + AHEAD <= whole; q0 += UNROLL) pieces<UNROLL>(piece, q0, std::false_type());
#pragma clang loop unroll(disable)
  for (; q0 < NS * PPS; q0 += UNROLL) pieces<UNROLL>(piece, q0, std::true_type(), NS * PPS);

  store_tile<A8, OUT_BF16, CF, MI>(p, t, acc, sm.ls, 0, colw + 4 * CF * grp, l15);
}

// ---------------------------------------------------------------- wide tiles
constexpr int kWideThreads = 512, kWideRows = 256, kWideCols = 256;

struct WideLds {
  static constexpr int NST = 4, B = 64;          // stages of one piece (128 elements); bytes of a row a stage
  uint8_t x[NST][kWideRows * B];
  uint8_t w[NST][kWideCols * B];
  uint8_t ws[2][kWideCols * kPitch];
  uint8_t xs[2][kWideRows * kPitch];
  int4 desc[kDesc];
};
static_assert(sizeof(WideLds) <= 160 * 1024, "LDS of a CU");

// Slot of chunk c of a staged row r of 64 bytes: c ^ its swizzle (two such rows share a 128-byte line).  Rows' fragments
// read 16 rows in a run; weights' lanes l%16 rows 16 (l%16 / 4) + l%4 (+ 4 f), eight neighbouring lanes two runs of
// four rows, 16 apart.
__device__ __forceinline__ int xswz64(int r) { return (r >> 1) & 3; }
__device__ __forceinline__ int wswz64(int r) { return ((r >> 1) & 1) + 2 * ((r >> 4) & 1); }

// One tile, up to 32 MI rows by 256 columns: two waves by four, each 16 MI rows by 64 columns.  Rows and weights
// both go to LDS by direct loads (neighbouring lanes on one row), NST - 1 stages ahead.  The fragments are plain LDS
// reads, which the compiler spreads over the products; their addresses are integers, since for a pointer into the
// array that the direct loads fill it would wait for every load in flight before each read.
template <bool OUT_BF16, int MI>
__device__ __forceinline__ void run_wide(const Mx4Args& p, WideLds& sm, const Tile& t) {
  constexpr int NST = WideLds::NST, B = WideLds::B;
  constexpr int ND = (MI + 3) / 4, NW = kWideCols * B / 8192, NL = ND + NW;          // a wave's loads a stage, 16 rows each
  const int tid = opaque(threadIdx.x);
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l15 = lane & 15, grp = lane >> 4, wr = wave >> 2, wc = wave & 3;
  const int kb = static_cast<int>(p.K / 32);
  const int bytes = static_cast<int>(p.K / 2);
  const int NS = (kb + 3) / 4, nwin = (kb + 15) / 16;

  // rows: wave w stages rows 4 MI w .. ; rows past the tile's last lie outside the buffer (zeros)
  const uint32_t ldl = static_cast<uint32_t>(p.ldl);
  const __amdgpu_buffer_rsrc_t xbuf = buffer(p.lhs + t.row0 * p.ldl, (t.rows - 1) * ldl + bytes);
  const int r0 = 4 * MI * wave + (lane >> 2);
  const uint32_t xoff = r0 * ldl;
  const int xc = 16 * ((lane & 3) ^ xswz64(r0));
  // weights: wave w stages rows 32 w .. 32 w + 31; columns past N lie outside the buffer (zeros, never stored)
  const int ncols = static_cast<int>(min(p.N - t.col0, static_cast<int64_t>(kWideCols)));
  const __amdgpu_buffer_rsrc_t wbuf =
      buffer(p.rhs + (static_cast<int64_t>(t.g) * p.N + t.col0) * bytes, static_cast<uint32_t>(ncols) * bytes);
  const int w0 = 32 * wave + (lane >> 2);        // and 16 more
  const uint32_t woff = static_cast<uint32_t>(w0) * bytes;
  const int wc0 = 16 * ((lane & 3) ^ wswz64(w0));
  auto load_stage = [&](int s, auto end_c) {
    uint8_t* xd = sm.x[s % NST] + 4 * MI * wave * B;
    uint8_t* wd = sm.w[s % NST] + 32 * wave * B;
    // chunks past a row's end: its last one (the weights there are zeroed before their use)
    const bool part = decltype(end_c)::value && B * s + B > bytes;
    const int last = part ? bytes - 16 - B * s : 64;
#pragma unroll
    for (int i = 0; i < NW; ++i) {               // 16 rows on: the other half of the swizzle
      const uint32_t c = min(wc0 ^ (32 * i), last);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wbuf, (lds_void*)(wd + 1024 * i), 16, woff + c, B * s + 16 * i * bytes, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < ND; ++i)
      if (16 * i + 16 <= 4 * MI || 16 * i + (lane >> 2) < 4 * MI)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_void*)(xd + 1024 * i), 16, xoff + min(xc, last), B * s + 16 * i * ldl, 0, 0);
  };

  const uint8_t* wsbase = p.rs + static_cast<int64_t>(t.g) * p.N * kb;
  const int col0 = static_cast<int>(t.col0);
  auto load_scales = [&](int win) {              // as in run_tile: five dwords a row and window
    const int ln = opaque(lane);
    const uint32_t ws_last = static_cast<uint32_t>(p.N * kb / 4 - 1);
    uint8_t* dst = sm.ws[win & 1] + wave * 32 * kPitch;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int idx = 64 * i + ln, r = idx / 5, d = idx - 5 * r;
      const uint32_t row = col0 + min(32 * wave + r, ncols - 1);
      const uint32_t dw = min((row * kb + 16 * win) / 4 + d, ws_last);
      if (r < 32) __builtin_amdgcn_global_load_lds(wsbase + 4 * dw, (lds_void*)(dst + 256 * i), 4, 0, 0);
    }
    {
      uint8_t* xd = sm.xs[win & 1] + wave * 4 * MI * kPitch;
      const uint8_t* base = static_cast<const uint8_t*>(p.ls) + t.row0 * p.lds;
      const int64_t end = (p.M - t.row0 - 1) * p.lds + ((kb + 3) & ~3) - 4;
#pragma unroll
      for (int i = 0; i < (20 * MI + 63) / 64; ++i) {
        const int idx = 64 * i + ln, r = idx / 5, d = idx - 5 * r;
        const int row = min(4 * MI * wave + r, t.rows - 1);
        const int64_t off = min(static_cast<int64_t>(row) * p.lds + 16 * win + 4 * d, end);
        if (r < 4 * MI) __builtin_amdgcn_global_load_lds(base + off, (lds_void*)(xd + 256 * i), 4, 0, 0);
      }
    }
  };

  v4f acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[i][f] = v4f{0.f, 0.f, 0.f, 0.f};

  step_barrier();                                // the last tile's readers are done
  load_scales(0);
  order();
#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (s < NS) load_stage(s, std::true_type());
  order();
  if (NS >= NST - 1)
    __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * NL));
  else
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));

  // fragment addresses in stage 0
  const int xr = 16 * MI * wr + l15, wrow = 64 * wc + 16 * (l15 >> 2) + (l15 & 3);   // weight row of fragment 0; 4 f more for f
  const uint32_t xa0 = lds_addr(sm.x[0]) + xr * B + 16 * (grp ^ xswz64(xr));
  const uint32_t xsa0 = lds_addr(sm.xs[0]) + xr * kPitch + grp;
  const uint32_t wa0 = lds_addr(sm.w[0]) + wrow * B + 16 * (grp ^ wswz64(wrow));
  const uint32_t wsa0 = lds_addr(sm.ws[0]) + wrow * kPitch + (static_cast<uint32_t>((col0 + wrow) * kb) & 3) + grp;

  auto stage = [&](int s, auto end_c) {
    constexpr bool END = decltype(end_c)::value;
    step_barrier();                              // every wave's loads of stage s are there; stage s - 1 is read
    if (s % 4 == 0 && s / 4 + 1 < nwin) load_scales(s / 4 + 1);
    order();
    if (!END || s + NST - 1 < NS) load_stage(s + NST - 1, end_c);
    order();
    const uint32_t win = (s / 4) & 1, sc = 4 * (s % 4);
    const uint32_t xb = xa0 + (s % NST) * static_cast<uint32_t>(sizeof(sm.x[0])), wb = wa0 + (s % NST) * static_cast<uint32_t>(sizeof(sm.w[0]));
    uint4 w[4];
    uint32_t ws[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {                // chunk l/16; rows 4 apart take the same swizzle
      w[f] = __builtin_bit_cast(uint4, lds_read<v4i>(wb + f * 4 * B));
      ws[f] = lds_read<uint8_t>(wsa0 + win * static_cast<uint32_t>(sizeof(sm.ws[0])) + sc + f * 4 * kPitch);
    }
    const bool past = END && 4 * s + grp >= kb;  // blocks past K: zero weights, plain scales for both operands
    if (END && s == NS - 1) {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        w[f].x = past ? 0 : w[f].x;
        w[f].y = past ? 0 : w[f].y;
        w[f].z = past ? 0 : w[f].z;
        w[f].w = past ? 0 : w[f].w;
        ws[f] = past ? 127 : ws[f];
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const v4i v = lds_read<v4i>(xb + 16 * B * i);
      const v8i x{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      uint32_t xs = lds_read<uint8_t>(xsa0 + win * static_cast<uint32_t>(sizeof(sm.xs[0])) + sc + 16 * kPitch * i);
      if (END) xs = past ? 127 : xs;
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[i][f] = mfma_mx4<false>(frag16(w[f]), ws[f], x, xs, acc[i][f]);
    }
    // this wave's loads of stage s + 1 have landed when only the later stages' are outstanding (in order; a scale
    // window is issued before the stage's)
    if (!END || s + NST - 1 < NS)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * NL));
    else
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  };
  int s = 0;
  // the furthest load, of stage s + NST - 1, is whole
  const int whole = static_cast<int>(p.K / 128);
#pragma clang loop unroll(disable)
  for (; s + NST <= whole; ++s) stage(s, std::false_type());
#pragma clang loop unroll(disable)
  for (; s < NS; ++s) stage(s, std::true_type());

  store_tile<false, OUT_BF16, 4, MI>(p, t, acc, nullptr, 16 * MI * wr, t.col0 + 64 * wc + 16 * grp, l15);
}

// Persistent workgroups (narrow: four waves, two a CU; wide: eight waves, one
// a CU).  A tile is up to 128 rows of one group by 64 columns, or 256 by 256
// (a group's rows are spread evenly over as few tiles as hold them); the tile range
// is split over the XCDs, row tiles fastest, so that a group's weights are
// fetched once and shared in L2.
template <bool A8, bool OUT_BF16, int CF>
__global__ __launch_bounds__(CF == 4 && !A8 ? kWideThreads : kThreads, 2) void gmm_mx4_kernel(const Mx4Args p) {
  constexpr bool WIDE = CF == 4 && !A8;
  using LDS = std::conditional_t<WIDE, WideLds, Lds<A8>>;
  __shared__ __attribute__((aligned(1024))) LDS sm;
  constexpr int BN = 64 * CF, THREADS = WIDE ? kWideThreads : kThreads;
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
    for (int g = tid; g < p.El; g += THREADS) {
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
    for (int g = tid; g < p.El; g += THREADS) gt.tmp[g] = row_tiles(gt.rows_off[g + 1] - gt.rows_off[g], p.tile_rows) * NT;
    __syncthreads();
    wave0_scan(gt.tmp, gt.tiles_off, p.El);
    __syncthreads();
    xcd_share(gt.tiles_off[p.El], first, last, step);
    n_rows = gt.rows_off[p.El];
    const int left = first < last ? (last - first + step - 1) / step - base : 0;       // this workgroup's tiles
    if (tid < min(left, kDesc)) {
      const int t = first + (base + tid) * step;
      const int g = find_group(gt, p.El, t);
      const int m = gt.rows_off[g + 1] - gt.rows_off[g], nb = row_tiles(m, p.tile_rows), fr = tile_frags(m, nb);
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
      const int blocks = (t.rows + 15) / 16;
      if constexpr (WIDE) {
        switch ((blocks + 1) / 2) {
          case 1: run_wide<OUT_BF16, 1>(p, sm, t); break;
          case 2: run_wide<OUT_BF16, 2>(p, sm, t); break;
          case 3: run_wide<OUT_BF16, 3>(p, sm, t); break;
          case 4: run_wide<OUT_BF16, 4>(p, sm, t); break;
          case 5: run_wide<OUT_BF16, 5>(p, sm, t); break;
          case 6: run_wide<OUT_BF16, 6>(p, sm, t); break;
          case 7: run_wide<OUT_BF16, 7>(p, sm, t); break;
          default: run_wide<OUT_BF16, 8>(p, sm, t);
        }
      } else {
        // (64 columns: an odd count of blocks above two runs as the next even one, which costs it little)
        constexpr bool ODD = CF == 4;
        if (blocks == 1) run_tile<A8, OUT_BF16, CF, 1>(p, sm, t);
        else if (blocks == 2) run_tile<A8, OUT_BF16, CF, 2>(p, sm, t);
        else if (blocks <= 4) {
          if (ODD && blocks == 3) run_tile<A8, OUT_BF16, CF, ODD ? 3 : 4>(p, sm, t);
          else run_tile<A8, OUT_BF16, CF, 4>(p, sm, t);
        } else if (blocks <= 6) {
          if (ODD && blocks == 5) run_tile<A8, OUT_BF16, CF, ODD ? 5 : 6>(p, sm, t);
          else run_tile<A8, OUT_BF16, CF, 6>(p, sm, t);
        } else {
          if (ODD && blocks == 7) run_tile<A8, OUT_BF16, CF, ODD ? 7 : 8>(p, sm, t);
          else run_tile<A8, OUT_BF16, CF, 8>(p, sm, t);
        }
      }
    }
    if (left <= kDesc) break;
  }
  // rows past the last group's are zero
  const int64_t bytes = (p.M - n_rows) * p.N * (OUT_BF16 ? 2 : 4);
  uint8_t* z = static_cast<uint8_t*>(p.out) + n_rows * p.N * (OUT_BF16 ? 2 : 4);
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * THREADS + opaque(threadIdx.x)) * 16; i < bytes;
       i += static_cast<int64_t>(gridDim.x) * THREADS * 16)
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
hipError_t launch(Mx4Args p, hipStream_t st) {
  // 256-column tiles when they fill the GPU's workgroups (4-bit rows: one a CU, e4m3: two), 64-column ones otherwise
  const int64_t groups = p.El < p.M ? p.El : p.M;
  const int64_t wide_rows = A8 ? kRows : kWideRows, wide_slots = (A8 ? 2 : 1) * num_cus();
  const bool wide = (groups + p.M / wide_rows) * moe_cdiv(p.N, 256) >= wide_slots;
  const int64_t slots = wide ? wide_slots : 2 * num_cus();
  const int64_t col_tiles = moe_cdiv(p.N, wide ? 256 : 64);
  // 64-column tiles: of half the rows as long as every one has a workgroup (512 ragged rows by 1040 columns: 15.1 us
  // with 64 rows, 18.2 with 128, 20.2 with 32)
  const bool half = !wide && (moe_cdiv(p.M, kRows / 2) + groups) * col_tiles <= slots;
  p.tile_rows = static_cast<int>(wide ? wide_rows : half ? kRows / 2 : kRows);
  const int64_t most = (moe_cdiv(p.M, p.tile_rows) + groups) * col_tiles;
  const unsigned grid = static_cast<unsigned>(most < 8 ? 8 : most < slots ? most : slots);   // each XCD's part has its own workgroups
  if (wide)
    gmm_mx4_kernel<A8, OUT_BF16, 4><<<grid, A8 ? kThreads : kWideThreads, 0, st>>>(p);
  else
    gmm_mx4_kernel<A8, OUT_BF16, 1><<<grid, kThreads, 0, st>>>(p);
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
      group_offset > E - num_local_experts)
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
                 group_sizes, group_offset, num_local_experts, M, K, N, out, static_cast<int32_t*>(ws), 0};
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
