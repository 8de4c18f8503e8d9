// moe_gmm_b128, moe_tgmm_b128: grouped products of e4m3 operands that share a
// scale over every 128 elements of the contraction, on the gfx950 scaled matrix
// cores (v_mfma_scale_f32_16x16x128_f8f6f4, float32 accumulate):
//   gmm    out[r, c] = sum_b sx[r, b] sw[g, b, c / 128] sum_{k in b} X[r, k] W_g[c, k]
//   tgmm   out[g, k, c] = sum_b sx[b, k] sy[b, c] sum_{r in b} Xt[b, k, r] Yt[b, c, r]
// One matrix instruction spans one block of the contraction, and its e8m0
// operands apply both scales: they cost nothing.
//
// An MFMA lane l supplies row l%16 of each operand, two 16-byte pieces of the
// 128: elements 16*(l/16) .. and 64 + 16*(l/16) .. (any share does, as both
// operands take the same and the scale is one for all).  The product is formed
// transposed per 16 x 16 block (the weights are the first operand), so output
// lane l holds row l%16 and four consecutive columns 4*(l/16) .. +3.
//
// Three kernels, by a rule on sizes alone (b128_rule.hpp):
//   few      few pieces of 16 rows (or up to 64) by 16 columns: every weight is met by a row or a few; latency and the
//            weights' bytes decide.  One row of 7168 x 4096: 8.6 us (29 MB, 3.4 TB/s).
//   wide     at least a tile for every workgroup: a 256 x 256 x 128 step takes 4050 clocks where its LDS reads take 1630, its
//            fill 512 and the matrix instructions 2048 (counters): they go in turn.  With operands in L2 3100 to 3450; with
//            float32 scales, 16 products of a sum with the change of units for every four matrix instructions, 5000.
//            32768 rows in 64 groups of 2048 x 1536, three tiles of 16 steps a workgroup: e8m0 134 us (1.5 PFLOP/s; 94 in steps,
//            25 in stores), float32 142; 8192 rows in 32 of 7168 x 4096: 271 us (1.8 PFLOP/s); 128 rows in 64 of
//            2048 x 1536: 43 us (4.2 TB/s of weights).  tgmm, 32768 rows in 64 groups, 4096 x 1536: bf16 results 290 to
//            300 us, of which 190 are left without the stores (0.8 GB, 118 us to a plain fill): they do not overlap; float32 400.
//   narrow   fewer tiles than that: the latency of a tile's stages.  512 ragged rows in 8 groups of 2080 x 1040: 12.5 us (wide
//            tiles 22); 256 rows in 32 groups of 4096 x 1536: 46 us (4.4 TB/s).
#include <type_traits>

#include "b128_common.hpp"
#include "b128_rule.hpp"
#include "stage_common.hpp"

namespace moe {
namespace {
using namespace tile;
using namespace stage;

enum Kind { kGmmE8M0, kGmmF32, kTgmm };

// What the calls accept, and the offsets inside a tile count on: K, N and the rows' stride; the stride of their scales.
constexpr int64_t kMaxLength = 1 << 22, kMaxScaleStride = 1 << 23;
// Offsets that lie outside every buffer: of a load, and of a store (whose buffers are larger).
constexpr uint32_t kNowhere = 0x80000000u, kNoStore = 0xf0000000u;

struct B128Args {
  const uint8_t* x;            // gmm: rows [M, K]; tgmm: [cols / 128, K, 128]
  int64_t ldx;
  const uint8_t* xs;           // gmm: [M, lds]; tgmm: [cols / 128, K]
  int64_t lds;
  const uint8_t* w;            // gmm: [El, N, K]; tgmm: [cols / 128, N, 128]
  const void* ws;              // gmm: [El, kb, nb]; tgmm: [cols / 128, N]
  const int32_t* sizes;
  int g0, El;
  int64_t M, K, N;
  void* out;
  int32_t* err;
};

// (Of the scale operands the lowest bytes.)
__device__ __forceinline__ v4f mfma_scaled(const v8i& w, uint32_t ws, const v8i& x, uint32_t xs, const v4f& c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, ws, 0, xs);
}

__device__ __forceinline__ v8i frag(const uint4& a, const uint4& b) {
  return v8i{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
             static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
}

// A float32 scale as a power of two, which the matrix core applies to the products' exponents, times a factor in [1, 2) with
// the scale's sign: no block's sum leaves float32's range where scale times sum stays in it.  What a subnormal lies below
// e8m0's smallest power comes off the rows' codes (by `down`; a code that would fall below 0 belongs to results that are 0
// in float32 either way), and a scale of 0 takes them all to the lowest: such a block adds nothing, or NaN for a NaN in it.
// A scale that is not finite is NaN.
struct F32Scale {
  uint32_t code, down;
  float factor;
};
__device__ __forceinline__ F32Scale split_scale(uint32_t v) {
  const uint32_t e = (v >> 23) & 255u, f = v & 0x7fffffu, lz = __builtin_clz(f | 1u);
  const uint32_t one = (v & 0x80000000u) | 0x3f800000u;
  if (e == 255u) return {255u, 0u, 1.0f};
  if (e != 0u) return {e, 0u, __uint_as_float(one | f)};
  if (f == 0u) return {0u, 255u, 1.0f};
  return {0u, lz - 9u, __uint_as_float(one | ((f << (lz - 8u)) & 0x7fffffu))};
}
__device__ __forceinline__ uint32_t lowered(uint32_t code, uint32_t down) {
  return code == 255u ? code : __builtin_elementwise_sub_sat(code, down);
}

// Two values to bfloat16, nearest even, in one operation (f32_to_bf16 takes eight for each).
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2bf));
}

template <bool OUT_BF16>
__device__ __forceinline__ void store4(void* out, int64_t at, const v4f& v) {
  if (OUT_BF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
}

// Rows past the last group's are zero.
template <bool OUT_BF16, int THREADS>
__device__ __forceinline__ void zero_rows(const B128Args& p, int64_t n_rows) {
  const int64_t bytes = (p.M - n_rows) * p.N * (OUT_BF16 ? 2 : 4);
  uint8_t* z = static_cast<uint8_t*>(p.out) + n_rows * p.N * (OUT_BF16 ? 2 : 4);
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x) * 16; i < bytes; i += static_cast<int64_t>(gridDim.x) * THREADS * 16)
    *reinterpret_cast<uint4*>(z + i) = make_uint4(0, 0, 0, 0);
}

// The local groups' rows and tiles (tgmm: blocks) of tiles with up to ROWS rows, for the kernels that decode tiles: in the
// stages' LDS, which is free while they do.
struct Table {
  int rows_off[kMaxLocal + 1], tiles_off[kMaxLocal + 1], blocks_off[kMaxLocal + 1], tmp[kMaxLocal];
};
template <Kind KIND, int ROWS>
__device__ __forceinline__ void group_table(const B128Args& p, Table& gt, int tid, int threads, int col_tiles) {
  for (int g = tid; g < p.El; g += threads) {
    int m = p.sizes[p.g0 + g];
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
  for (int g = tid; g < p.El; g += threads) {
    const int m = gt.rows_off[g + 1] - gt.rows_off[g];
    gt.tmp[g] = KIND == kTgmm ? (m + 127) / 128 : row_tiles(m, ROWS) * col_tiles;
  }
  __syncthreads();
  wave0_scan(gt.tmp, KIND == kTgmm ? gt.blocks_off : gt.tiles_off, p.El);
  __syncthreads();
}

// Tile t: first row (tgmm: in the group's result), column tile, group, rows; blocks of the contraction, first block.
template <Kind KIND, int ROWS>
__device__ __forceinline__ void decode_tile(const B128Args& p, const Table& gt, int t, int row_tiles_tgmm, int col_tiles, int4& desc, int2& more) {
  if (KIND == kTgmm) {
    const int g = t / (row_tiles_tgmm * col_tiles), l = t - g * row_tiles_tgmm * col_tiles, rt = l / col_tiles, ct = l - rt * col_tiles;
    desc = make_int4(ROWS * rt, ct, g, min(ROWS, static_cast<int>(p.K) - ROWS * rt));
    more = make_int2(gt.blocks_off[g + 1] - gt.blocks_off[g], gt.blocks_off[g]);
  } else {
    const int g = find_group(gt, p.El, t);
    const int m = gt.rows_off[g + 1] - gt.rows_off[g], nr = row_tiles(m, ROWS), fr = tile_frags(m, nr);
    const int local = t - gt.tiles_off[g], ct = local / nr, rt = local - ct * nr;
    // (even filling may leave a last tile without rows: it has no stages)
    const int rows = max(min(16 * fr, m - 16 * fr * rt), 0);
    desc = make_int4(gt.rows_off[g] + 16 * fr * rt, ct, g, rows);
    more = make_int2(rows ? static_cast<int>((p.K + 127) / 128) : 0, 0);
  }
}

// ---------------------------------------------------------------- few rows
// 16 MI rows by 16 columns a workgroup: the weights of sixteen columns are a
// stream of K bytes each, its blocks dealt out to eight waves, a wave's loads of
// several blocks issued before their products, and the waves' sums added in wave
// order.  For decoding: every weight is met by a row or a few, and what counts is to
// have its bytes under way at once.
constexpr int kSplit = 8;

template <Kind KIND, bool OUT_BF16, int MI>
__global__ __launch_bounds__(64 * kSplit) void b128_few_kernel(const B128Args p, int tiles) {
  constexpr int AHEAD = MI == 1 ? 8 : MI == 2 ? 4 : 2;                   // blocks loaded before their products
  __shared__ v4f part[kSplit][MI][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l15 = lane & 15, grp = lane >> 4;
  const int NT = static_cast<int>(p.N / 16), M = static_cast<int>(p.M);
  const int j = blockIdx.x / NT, ct = blockIdx.x - j * NT;
  int g = 0, row0 = 16 * MI * j, rows, there;      // the tile's group and rows; rows that there are to load
  if (p.El == 1) {                                 // nothing but the store waits for the size
    const int m = p.sizes[p.g0];
    if (blockIdx.x == 0 && tid == 0 && m < 0) raise_error(p.err, MOE_DEVERR_GROUP_SIZE);
    if (blockIdx.x == 0 && tid == 0 && m > M) raise_error(p.err, MOE_DEVERR_ROWS);
    rows = min(m, M) - row0;
    there = M - row0;
  } else {                                         // the group that holds row tile j, of `tiles` - 1 at most
    const bool tell = j == tiles - 1 && ct == 0 && wave == 0;            // (the last tile is nobody's: it meets every size)
    int have = 0, before = 0;
    bool found = false;
    for (int base = 0; base < p.El && !found; base += 64) {
      const int raw = base + lane < p.El ? p.sizes[p.g0 + base + lane] : 0;
      const int end = b128::wave_scan(min(min(max(raw, 0), M) + (lane == 0 ? have : 0), M), M);      // rows up to this group's last
      const int up = __builtin_amdgcn_update_dpp(have, end, 0x138, 0xf, 0xf, false);                 // wave_shr 1: up to its first
      if (tell && raw < 0) raise_error(p.err, MOE_DEVERR_GROUP_SIZE);
      if (tell && raw > M - up) raise_error(p.err, MOE_DEVERR_ROWS);
      const int n = (end - up + 16 * MI - 1) / (16 * MI), last = before + b128::wave_scan(n, M);
      const uint64_t has = __ballot(last > j);
      if (has) {
        const int l = __builtin_ctzll(has), at = 16 * MI * (j - __builtin_amdgcn_readlane(last - n, l));
        found = true;
        g = base + l;
        row0 = __builtin_amdgcn_readlane(up, l) + at;
        rows = __builtin_amdgcn_readlane(end - up, l) - at;
      }
      have = __builtin_amdgcn_readlane(end, 63);
      before = __builtin_amdgcn_readlane(last, 63);
    }
    if (!found) {                                  // rows past the last group's are zero
      if (j == tiles - 1)
        for (int i = tid; i < 4 * (M - have); i += 64 * kSplit) store4<OUT_BF16>(p.out, (have + (i >> 2)) * p.N + 16 * ct + 4 * (i & 3), v4f{0.f, 0.f, 0.f, 0.f});
      return;
    }
    there = rows;
  }
  const uint32_t K = static_cast<uint32_t>(p.K), ldx = static_cast<uint32_t>(p.ldx);
  const int kb = static_cast<int>((K + 127) / 128), nb = static_cast<int>((p.N + 127) / 128);
  const __amdgpu_buffer_rsrc_t xbuf = buffer(p.x + row0 * p.ldx, (min(there, 16 * MI) - 1) * ldx + K);
  const __amdgpu_buffer_rsrc_t wbuf = buffer(p.w + (static_cast<int64_t>(g) * p.N + 16 * ct) * p.K, 16 * K);
  const uint8_t* xs = p.xs + (row0 + static_cast<int64_t>(min(l15, there - 1))) * p.lds;
  const int64_t ws0 = static_cast<int64_t>(g) * kb * nb + ct / 8;
  v4f acc[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const int per = (kb + kSplit - 1) / kSplit, end = min(kb, (wave + 1) * per);
  for (int b0 = wave * per; b0 < end; b0 += AHEAD) {
    uint4 w[AHEAD][2], x[AHEAD][MI][2];
    uint32_t xsc[AHEAD][MI], wsc[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (b0 + u >= end) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {                // chunks past K, and rows past those there are, lie outside the buffers: zeros
        const uint32_t at = 128u * (b0 + u) + 64 * h + 16 * grp, o = at < K ? at : kNowhere;
        w[u][h] = buffer_load16(wbuf, l15 * K + o, 0);
#pragma unroll
        for (int i = 0; i < MI; ++i) x[u][i][h] = buffer_load16(xbuf, (16 * i + l15) * ldx + o, 0);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) xsc[u][i] = 16 * i + l15 < there ? xs[16 * i * p.lds + b0 + u] : 0;
      const int64_t at = ws0 + static_cast<int64_t>(b0 + u) * nb;
      if (KIND == kGmmF32)
        wsc[u] = static_cast<const uint32_t*>(p.ws)[at];
      else
        wsc[u] = static_cast<const uint8_t*>(p.ws)[at];
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (b0 + u >= end) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const v8i wv = frag(w[u][0], w[u][1]), xv = frag(x[u][i][0], x[u][i][1]);
        if constexpr (KIND == kGmmF32) {
          const F32Scale sc = split_scale(wsc[u]);
          acc[i] += sc.factor * mfma_scaled(wv, sc.code, xv, lowered(xsc[u][i], sc.down), v4f{0.f, 0.f, 0.f, 0.f});
        } else
          acc[i] = mfma_scaled(wv, wsc[u], xv, xsc[u][i], acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  const int r = 16 * wave + l15;
  if (wave < MI && r < (p.El == 1 ? there : rows)) {
    v4f sum = part[0][wave][lane];
#pragma unroll
    for (int i = 1; i < kSplit; ++i) sum += part[i][wave][lane];
    if (r >= rows) sum = v4f{0.f, 0.f, 0.f, 0.f};
    store4<OUT_BF16>(p.out, (row0 + static_cast<int64_t>(r)) * p.N + 16 * ct + 4 * grp, sum);
  }
}

// ---------------------------------------------------------------- wide tiles
// Up to 320 x 256 results a workgroup of eight waves, two by four, each 16 MI rows
// by 64 columns.  A stage is one block of the contraction, 128 bytes of every
// row of both operands (whole lines), by direct loads to LDS, two stages of each.
// A wave reads its weights of a stage at the stage's start; behind the barrier that
// follows, the weights two stages on take their place, while the rows of the next
// stage have been on their way since its start.  The stream runs on from tile to
// tile, under the stores of the last one's results.
constexpr int kWideThreads = 512, kWindow = 16, kDesc = 64;
using b128::kNarrow;
using b128::kWideCols;
template <Kind KIND>
constexpr int kWideRows = KIND == kTgmm ? b128::kWideRowsTgmm : b128::kWideRowsGmm;

template <Kind KIND>
struct WideLds {
  uint8_t x[2][kWideRows<KIND> * 128];
  uint8_t w[2][kWideCols * 128];
  uint8_t xs[2][kWideRows<KIND> * kWindow];        // scales of a window of 16 blocks: gmm a row's 16 bytes, tgmm a block's 256
  uint8_t ws[2][KIND == kTgmm ? kWideCols * kWindow : 8 * kWindow];    // gmm: 16 blocks by 2, a dword each
  int4 desc[kDesc];                                // first row, column tile, group, rows
  int2 more[kDesc];                                // blocks, first block
};
static_assert(kWideRows<kGmmE8M0> * kMaxLength <= kNowhere && kWideCols * kMaxLength <= kNowhere &&
              kWideRows<kGmmE8M0> * kMaxScaleStride < (int64_t{1} << 32), "offsets of a tile's operands");
static_assert(sizeof(WideLds<kGmmE8M0>) <= 160 * 1024 && sizeof(WideLds<kTgmm>) <= 160 * 1024, "LDS of a CU");

// Slot of 16-byte chunk c of a staged row r: c ^ swizzle(r).  Rows of even and odd number lie in different halves of
// the banks; of the sixteen rows that a read's neighbouring lanes are at, the eight of either kind lie in eight slots:
// runs of rows, or (bf16 results) lanes l%16 at rows 8 (l%16 / 4) + l%4.
__device__ __forceinline__ int swz_run(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int swz_quads(int r) { return ((r & 3) + 4 * ((r >> 3) & 1)) ^ ((r >> 4) & 1); }
// First column in a wave's 64 of what lane l%16 = n supplies as weight row of fragment f: output lanes l/16 then hold
// columns whose stores make runs of 64 bytes, eight bf16 of fragments 2 h and 2 h + 1, or four float32 of one.
template <bool OUT_BF16>
__device__ __forceinline__ constexpr int frag_col(int f, int n) {
  return OUT_BF16 ? 32 * (f >> 1) + 8 * (n >> 2) + 4 * (f & 1) + (n & 3) : 16 * f + n;
}

struct WideTile {
  int row0, col0;                                  // (tgmm: in the group's result)
  int g, rows, steps, blk0;
};

template <class LDS>
__device__ __forceinline__ WideTile wide_tile(const LDS& sm, int i) {
  const v4i d = lds_read<v4i>(lds_addr(sm.desc) + 16 * i);
  const v2i m = lds_read<v2i>(lds_addr(sm.more) + 8 * i);
  WideTile t;
  t.row0 = __builtin_amdgcn_readfirstlane(d[0]);
  t.col0 = __builtin_amdgcn_readfirstlane(d[1]) * kWideCols;
  t.g = __builtin_amdgcn_readfirstlane(d[2]);
  t.rows = __builtin_amdgcn_readfirstlane(d[3]);
  t.steps = __builtin_amdgcn_readfirstlane(m[0]);
  t.blk0 = __builtin_amdgcn_readfirstlane(m[1]);
  return t;
}

// One operand's loads: where they are in the stream of tiles and stages, and to which buffer the next goes.
template <Kind KIND, bool OUT_BF16, bool ROWS>
struct Cursor {
  __amdgpu_buffer_rsrc_t buf;                      // gmm: the tile's
  const uint8_t* src;                              // tgmm: the stage's, which is one run of bytes
  WideTile t;
  int i, s, b;                                     // tile, stage, buffer
  bool more;                                       // whether there is such a stage

  // The first tile from i on that has stages.
  __device__ __forceinline__ void seek(const B128Args& p, const WideLds<KIND>& sm, int count) {
    s = 0;
    for (; i < count; ++i) {
      t = wide_tile(sm, i);
      if (t.steps > 0) break;
    }
    more = i < count;
    if (!more) return;
    if constexpr (KIND == kTgmm) {
      src = ROWS ? p.x + 128 * (t.blk0 * p.K + t.row0) : p.w + 128 * (t.blk0 * p.N + t.col0);
    } else {
      const uint32_t K = static_cast<uint32_t>(p.K), cols = static_cast<uint32_t>(min(static_cast<int>(p.N) - t.col0, kWideCols));
      buf = ROWS ? buffer(p.x + static_cast<int64_t>(t.row0) * p.ldx, (t.rows - 1) * static_cast<uint32_t>(p.ldx) + K)
                 : buffer(p.w + (static_cast<int64_t>(t.g) * p.N + t.col0) * p.K, cols * K);
    }
  }

  // The stage at hand; lane l fills slot l%8 of rows 8 wave + l/8 (+ 64 j).  Rows past the tile's, columns past N and
  // chunks past K lie outside the buffer: zeros.  (Weights are four loads always: the waits count them.)
  __device__ __forceinline__ void load(const B128Args& p, WideLds<KIND>& sm, int count, int wave, int lane) {
    const int r = 8 * wave + (lane >> 3);
    const uint32_t ld = KIND == kTgmm ? 128u : static_cast<uint32_t>(ROWS ? p.ldx : p.K);
    if constexpr (KIND == kTgmm) {
      buf = buffer(src, 128u * static_cast<uint32_t>(ROWS ? t.rows : min(static_cast<int>(p.N) - t.col0, kWideCols)));
      src += 128 * (ROWS ? p.K : p.N);
    }
    const uint32_t stage_at = KIND == kTgmm ? 0u : 128u * s;
    const uint32_t c = 16 * ((lane & 7) ^ (ROWS || !OUT_BF16 ? swz_run(r) : swz_quads(r)));
    uint32_t off = r * ld + c;
    if (KIND != kTgmm && 128 * s + 128 > p.K) off = c < static_cast<uint32_t>(p.K) - 128u * s ? off : kNowhere;
    uint8_t* dst = (ROWS ? sm.x[b] : sm.w[b]) + 8 * wave * 128;
#pragma unroll
    for (int j = 0; j < (ROWS ? kWideRows<KIND> : kWideCols) / 64; ++j)
      if (!ROWS || KIND == kTgmm || 64 * j + 8 * wave < t.rows)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void*)(dst + 64 * 128 * j), 16, off, stage_at + 64 * j * ld, 0, 0);
    b ^= 1;
    if (++s == t.steps) {
      ++i;
      seek(p, sm, count);
    }
  }
};

// Scales of blocks 16 n .. of tile t to window buffer `win`.  (What lies past the tile or the contraction is some scale or
// zero, and not used.  Buffer loads, as for the stages: behind a global load to LDS the compiler takes LDS reads to
// come back in any order, and waits for all of them at each use.)
template <Kind KIND>
__device__ __forceinline__ void load_scales(const B128Args& p, WideLds<KIND>& sm, const WideTile& t, int n, int win, int wave, int lane) {
  if constexpr (KIND == kTgmm) {                   // [block][K or N]: lanes 16 j .. 16 j + 15 the 256 bytes of block 4 wave + j
    const bool x = wave < 4;
    const int64_t len = x ? p.K : p.N, c = x ? t.row0 : t.col0;
    const uint8_t* src = (x ? p.xs : static_cast<const uint8_t*>(p.ws)) + (t.blk0 + static_cast<int64_t>(kWindow) * n) * len + c;
    const __amdgpu_buffer_rsrc_t buf = buffer(src, static_cast<uint32_t>(min(t.steps - kWindow * n, kWindow) * len - c));
    uint8_t* dst = (x ? sm.xs[win] : sm.ws[win]) + 1024 * (wave & 3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void*)dst, 16, (4 * (wave & 3) + (lane >> 4)) * static_cast<uint32_t>(len) + 16 * (lane & 15), 0, 0, 0);
  } else {
    constexpr int R = kWideRows<KIND> / 8;
    if (lane < R && R * wave < t.rows) {
      const uint32_t lds = static_cast<uint32_t>(p.lds);
      const __amdgpu_buffer_rsrc_t buf = buffer(p.xs + t.row0 * p.lds, t.rows * lds);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void*)(sm.xs[win] + R * kWindow * wave), 16, (R * wave + lane) * lds, kWindow * n, 0, 0);
    }
    if (wave == 7 && lane < 2 * kWindow) {         // block 16 n + lane / 2, column block lane & 1 of the tile's two
      const int nb = static_cast<int>((p.N + 127) / 128), size = KIND == kGmmF32 ? 4 : 1;
      const uint8_t* src = static_cast<const uint8_t*>(p.ws) + static_cast<int64_t>(t.g) * t.steps * nb * size;
      const uint32_t odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src)) & 3;       // (e8m0: the dword that holds the byte)
      const __amdgpu_buffer_rsrc_t buf = buffer(src - odd, (static_cast<uint32_t>(t.steps * nb * size) + odd + 3) & ~3u);
      const int at = (kWindow * n + (lane >> 1)) * nb + min(t.col0 / 128 + (lane & 1), nb - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void*)sm.ws[win], 4, (at * size + odd) & ~3u, 0, 0, 0);
    }
  }
}

// Every store is issued whatever the tile holds (rows past it, columns past N lie outside the buffer), so that their
// number is known to the waits.
template <Kind KIND, bool OUT_BF16, int MI>
__device__ __forceinline__ void wide_store(const B128Args& p, const WideTile& t, int wave, int lane, const v4f (&acc)[MI][4], float scale) {
  constexpr int B = OUT_BF16 ? 2 : 4;
  const int l15 = lane & 15, grp = lane >> 4, wr = wave >> 2, wc = wave & 3;
  const uint32_t ld = static_cast<uint32_t>(p.N) * B;
  const int64_t c = t.col0 + 64 * wc, row0 = (KIND == kTgmm ? t.g * p.K + t.row0 : t.row0) + 16 * MI * wr;
  const int rows = min(t.rows - 16 * MI * wr, 16 * MI);    // the wave's rows (or none)
  // 32 bits hold every offset, and no buffer reaches the stores that go nowhere (of the whole tile's rows it would)
  static_assert(16 * MI * kMaxLength * B + 64 * B <= kNoStore, "offsets of a wave's results");
  const int64_t left = p.N - c;                    // its columns
  const __amdgpu_buffer_rsrc_t o = buffer(static_cast<uint8_t*>(p.out) + (row0 * p.N + c) * B,
                                          rows > 0 && left > 0 ? (rows - 1) * ld + static_cast<uint32_t>(min(left, static_cast<int64_t>(64))) * B : 0u);
  const bool odd = l15 & 1;
  // A lane's two pieces of 16 bytes lie in the two halves of a line of its row.  Neighbouring lanes exchange one, so that a
  // store writes eight whole lines, of the even lanes' rows and then of the odd ones' (halves of sixteen: weight gradient
  // 470 us instead of 427, as the L2 takes them).
  auto put = [&](const v4u32& c0, const v4u32& c1, uint32_t row, int col) {
    v4u32 a, b;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t other = __builtin_amdgcn_update_dpp(0, odd ? c0[q] : c1[q], 0xb1, 0xf, 0xf, true);    // quad_perm [1, 0, 3, 2]
      a[q] = odd ? other : c0[q];
      b[q] = odd ? c1[q] : other;
    }
    const bool in = col < left;
    __builtin_amdgcn_raw_buffer_store_b128(a, o, in ? row + B * col : kNoStore, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(b, o, in ? row + ld + B * col : kNoStore, 0, 0);
  };
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const uint32_t row = (16 * i + (l15 & 14)) * ld;
    v4f v[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) v[f] = KIND == kGmmF32 ? acc[i][f] * scale : acc[i][f];
    if (OUT_BF16) {
      v4u32 u[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f& a = v[2 * h + (q >> 1)];
          u[h][q] = pack_bf16(a[2 * (q & 1)], a[2 * (q & 1) + 1]);
        }
      put(u[0], u[1], row, (odd ? 32 : 0) + 8 * grp);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        put(__builtin_bit_cast(v4u32, v[2 * h]), __builtin_bit_cast(v4u32, v[2 * h + 1]), row, 32 * h + (odd ? 16 : 0) + 4 * grp);
    }
  }
}

// Where a workgroup is in its tiles.
template <Kind KIND, bool OUT_BF16>
struct Stream {
  Cursor<KIND, OUT_BF16, true> x;
  Cursor<KIND, OUT_BF16, false> w;
  int count;
  int b, win;                                      // buffers of the stage at hand
  bool ahead;                                      // whether weights were issued behind the rows that are waited for

  // The next rows, and with a window's first its scales (to the window that is not in use).
  __device__ __forceinline__ void load_rows(const B128Args& p, WideLds<KIND>& sm, int to, int wave, int lane) {
    if (!x.more) return;
    if (x.s % kWindow == 0) load_scales<KIND>(p, sm, x.t, x.s / kWindow, to, wave, lane);
    x.load(p, sm, count, wave, lane);
  }
};

template <int I, int END, class F>
__device__ __forceinline__ void blocks(const F& f) {
  if constexpr (I < END) {
    f(std::integral_constant<int, I>());
    blocks<I + 1, END>(f);
  }
}

// One tile.
template <Kind KIND, bool OUT_BF16, int MI>
__device__ __forceinline__ void run_wide(const B128Args& p, WideLds<KIND>& sm, Stream<KIND, OUT_BF16>& st, const WideTile& t, bool stored) {
  constexpr int kStores = (OUT_BF16 ? 2 : 4) * MI;
  const int tid = opaque(threadIdx.x);
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l15 = lane & 15, grp = lane >> 4, wr = wave >> 2, wc = wave & 3;
  const int xr = 16 * MI * wr + l15, wrow = 64 * wc + frag_col<OUT_BF16>(0, l15);
  const uint32_t xa0 = lds_addr(sm.x[0]) + xr * 128 + 16 * (grp ^ swz_run(l15));
  const uint32_t wa0 = lds_addr(sm.w[0]) + wrow * 128 + 16 * (grp ^ (OUT_BF16 ? swz_quads(wrow) : swz_run(wrow)));
  v4f acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[i][f] = v4f{0.f, 0.f, 0.f, 0.f};
  uint32_t xsd[MI];                                // scales of the rows; gmm: four blocks of each, tgmm: one
  float unit = 1.0f;                               // float32 scales: what the sums are in units of
#pragma clang loop unroll(disable)
  for (int s = 0; s < t.steps; ++s) {
    // this wave's loads of the stage are there: the weights of the next may be on their way, and a tile's stores
    if (!st.ahead)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    else if (KIND == kTgmm && s == 0 && stored)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(4 + kStores));
    else
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(4));
    step_barrier();                                // every wave's are; the other buffer of rows is read
    const bool last_of_window = (s + 1) % kWindow == 0 || s + 1 == t.steps;
    st.load_rows(p, sm, st.win ^ 1, wave, lane);
    order();
    const uint32_t xa = xa0 + st.b * static_cast<uint32_t>(sizeof(sm.x[0])), wa = wa0 + st.b * static_cast<uint32_t>(sizeof(sm.w[0]));
    const uint32_t xsb = lds_addr(sm.xs[0]) + st.win * static_cast<uint32_t>(sizeof(sm.xs[0]));
    const uint32_t wsb = lds_addr(sm.ws[0]) + st.win * static_cast<uint32_t>(sizeof(sm.ws[0]));
    const int sb = s & (kWindow - 1);
    auto read_x = [&](int i) {
      return frag(__builtin_bit_cast(uint4, lds_read<v4i>(xa + 2048 * i)), __builtin_bit_cast(uint4, lds_read<v4i>((xa ^ 64u) + 2048 * i)));
    };
    v8i w[4];
    uint32_t wsc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const uint32_t at = frag_col<OUT_BF16>(f, 0) * 128;
      w[f] = frag(__builtin_bit_cast(uint4, lds_read<v4i>(wa + at)), __builtin_bit_cast(uint4, lds_read<v4i>((wa ^ 64u) + at)));
      if (KIND == kTgmm) wsc[f] = lds_read<uint8_t>(wsb + 256 * sb + wrow + frag_col<OUT_BF16>(f, 0));
    }
    v8i x[2];
    x[0] = read_x(0);
    if constexpr (KIND == kTgmm) {
#pragma unroll
      for (int i = 0; i < MI; ++i) xsd[i] = lds_read<uint8_t>(xsb + 256 * sb + xr + 16 * i);
    } else if ((sb & 3) == 0) {
#pragma unroll
      for (int i = 0; i < MI; ++i) xsd[i] = lds_read<uint32_t>(xsb + (xr + 16 * i) * kWindow + sb);
    }
    float ratio = 1.0f;
    if constexpr (KIND == kGmmE8M0) {
      const uint32_t nb = static_cast<uint32_t>((p.N + 127) / 128), c = min(static_cast<uint32_t>(t.col0) / 128 + (wc >> 1), nb - 1);
      const uint32_t byte = (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.ws)) + (static_cast<uint32_t>(t.g) * t.steps + s) * nb + c) & 3;
      wsc[0] = wsc[1] = wsc[2] = wsc[3] = lds_read<uint8_t>(wsb + 8 * sb + 4 * (wc >> 1) + byte);
    }
    const uint32_t shift = KIND == kTgmm ? 0 : 8 * (sb & 3);
    if constexpr (KIND == kGmmF32) {
      // The sums are held in units of the last block's factor, and change units by the ratio of two.
      const F32Scale sc = split_scale(__builtin_amdgcn_readfirstlane(lds_read<uint32_t>(wsb + 8 * sb + 4 * (wc >> 1))));
      if (s > 0) ratio = unit / sc.factor;
      unit = sc.factor;
      wsc[0] = wsc[1] = wsc[2] = wsc[3] = sc.code;
      if (sc.down) {                               // (rare: the stage's codes of the rows, in their places)
#pragma unroll
        for (int i = 0; i < MI; ++i) xsd[i] = (xsd[i] & ~(255u << shift)) | lowered((xsd[i] >> shift) & 255u, sc.down) << shift;
      }
    }
    auto block = [&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      if (i + 1 < MI) x[(i + 1) & 1] = read_x(i + 1);
      __builtin_amdgcn_sched_barrier(0);           // (left free, the compiler reads each block's rows behind the last one's products)
      if constexpr (KIND == kGmmF32) {
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[i][f] *= ratio;
      }
      const uint32_t xs = xsd[i] >> shift;
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[i][f] = mfma_scaled(w[f], wsc[f], x[i & 1], xs, acc[i][f]);
      __builtin_amdgcn_sched_barrier(0);
    };
    step_barrier();                                // every wave's weights are read
    if (st.w.more) {
      st.w.load(p, sm, st.count, wave, lane);
      st.ahead = true;
    } else {
      st.ahead = false;
    }
    order();
    blocks<0, MI>(block);
    st.b ^= 1;
    if (last_of_window) st.win ^= 1;
  }
  wide_store<KIND, OUT_BF16, MI>(p, t, wave, lane, acc, unit);
}

// Persistent workgroups, one a CU.  A group's rows are spread evenly over as few tiles as hold them; the tile range is
// split over the XCDs, row tiles (tgmm: column tiles) fastest, so that a group's weights are fetched once and shared in L2.
template <Kind KIND, bool OUT_BF16>
__global__ __launch_bounds__(kWideThreads, 2) void b128_wide_kernel(const B128Args p) {
  __shared__ __attribute__((aligned(1024))) WideLds<KIND> sm;
  constexpr bool TG = KIND == kTgmm;
  constexpr int ROWS = kWideRows<KIND>;
  const int NT = static_cast<int>((p.N + kWideCols - 1) / kWideCols), RT = TG ? static_cast<int>((p.K + ROWS - 1) / ROWS) : 0;
  // tiles are decoded up to kDesc at a time
  static_assert(sizeof(Table) <= sizeof(sm.x), "the group table fits the stages");
  Table& gt = *reinterpret_cast<Table*>(&sm.x[0][0]);
  int first = 0, last = 0, step = 1, n_rows = 0;
#pragma clang loop unroll(disable)
  for (int base = 0;; base += kDesc) {
    const int tid = opaque(threadIdx.x);
    __syncthreads();
    group_table<KIND, ROWS>(p, gt, tid, kWideThreads, NT);
    xcd_share(TG ? p.El * RT * NT : gt.tiles_off[p.El], first, last, step);
    n_rows = gt.rows_off[p.El];
    const int left = first < last ? (last - first + step - 1) / step - base : 0;       // this workgroup's tiles
    const int count = min(left, kDesc);
    if (tid < count) decode_tile<KIND, ROWS>(p, gt, first + (base + tid) * step, RT, NT, sm.desc[tid], sm.more[tid]);
    __syncthreads();
    if (count > 0) {
      const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
      Stream<KIND, OUT_BF16> st;
      st.count = count;
      st.b = st.win = 0;
      st.x.i = st.x.b = st.w.i = st.w.b = 0;
      st.x.seek(p, sm, count);
      st.w.seek(p, sm, count);
      if (st.w.more) st.w.load(p, sm, count, wave, lane);
      order();
      st.load_rows(p, sm, 0, wave, lane);
      order();
      st.ahead = st.w.more;
      if (st.w.more) st.w.load(p, sm, count, wave, lane);
      order();
#pragma clang loop unroll(disable)
      for (int i = 0; i < count; ++i) {
        const WideTile t = wide_tile(sm, i);
        if constexpr (TG) {
          run_wide<KIND, OUT_BF16, 8>(p, sm, st, t, i > 0);
        } else {
          switch ((t.rows + 31) / 32) {
            case 0: break;
            case 1: run_wide<KIND, OUT_BF16, 1>(p, sm, st, t, false); break;
            case 2: run_wide<KIND, OUT_BF16, 2>(p, sm, st, t, false); break;
            case 3: run_wide<KIND, OUT_BF16, 3>(p, sm, st, t, false); break;
            case 4: run_wide<KIND, OUT_BF16, 4>(p, sm, st, t, false); break;
            case 5: run_wide<KIND, OUT_BF16, 5>(p, sm, st, t, false); break;
            case 6: run_wide<KIND, OUT_BF16, 6>(p, sm, st, t, false); break;
            case 7: run_wide<KIND, OUT_BF16, 7>(p, sm, st, t, false); break;
            case 8: run_wide<KIND, OUT_BF16, 8>(p, sm, st, t, false); break;
            case 9: run_wide<KIND, OUT_BF16, 9>(p, sm, st, t, false); break;
            default: run_wide<KIND, OUT_BF16, 10>(p, sm, st, t, false);
          }
        }
      }
    }
    if (left <= kDesc) break;
  }
  if constexpr (!TG) zero_rows<OUT_BF16, kWideThreads>(p, n_rows);
}

// ---------------------------------------------------------------- narrow tiles
// 64 x 64 results a workgroup of eight waves, four by two, each 16 rows by 32
// columns; eight stages of both operands in LDS, seven ahead, the stream running on from
// tile to tile: for fewer rows or tiles than the wide ones fill the GPU with, where
// the loads' latency is the time.  Each stage brings its scales.
// Fewer than one wide tile a workgroup are fewer than 20 narrow ones (gmm: 64 rows for 320, 64 columns for 256, and a group's
// last tile; tgmm: 16), so at most 24 after the split over the XCDs, 42 on a device of 15 CUs.
constexpr int kNarrowStages = 8, kNarrowDesc = 64;

struct NarrowLds {
  uint8_t x[kNarrowStages][kNarrow * 128];
  uint8_t w[kNarrowStages][kNarrow * 128];
  uint32_t xs[kNarrowStages][kNarrow];             // gmm: the dword of each row that holds the block's byte; tgmm: 64 bytes
  uint32_t ws[kNarrowStages][kNarrow];             // gmm: one dword; tgmm: 64 bytes
  int4 desc[kNarrowDesc];                          // first row, column tile, group, rows
  int2 more[kNarrowDesc];                          // blocks, first block
};
static_assert(sizeof(NarrowLds) <= 160 * 1024, "LDS of a CU");

__device__ __forceinline__ WideTile narrow_tile(const NarrowLds& sm, int i) {
  WideTile t = wide_tile(sm, i);
  t.col0 = t.col0 / kWideCols * kNarrow;
  return t;
}

template <Kind KIND, bool OUT_BF16>
__global__ __launch_bounds__(kWideThreads, 2) void b128_narrow_kernel(const B128Args p) {
  __shared__ __attribute__((aligned(1024))) NarrowLds sm;
  constexpr bool TG = KIND == kTgmm;
  constexpr int NST = kNarrowStages;
  const int NT = static_cast<int>((p.N + kNarrow - 1) / kNarrow), RT = TG ? static_cast<int>((p.K + kNarrow - 1) / kNarrow) : 0;
  static_assert(sizeof(Table) <= sizeof(sm.x), "the group table fits the stages");
  Table& gt = *reinterpret_cast<Table*>(&sm.x[0][0]);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l15 = lane & 15, grp = lane >> 4, wr = wave >> 1, wc = wave & 1;
  const int nb = static_cast<int>((p.N + 127) / 128);
  group_table<KIND, kNarrow>(p, gt, tid, kWideThreads, NT);
  int first, last, step;
  xcd_share(TG ? p.El * RT * NT : gt.tiles_off[p.El], first, last, step);
  const int n_rows = gt.rows_off[p.El];
  const int count = first < last ? (last - first + step - 1) / step : 0;               // this workgroup's tiles
  if (tid < count) decode_tile<KIND, kNarrow>(p, gt, first + tid * step, RT, NT, sm.desc[tid], sm.more[tid]);
  __syncthreads();
  // the loads' place in the stream
  WideTile lt{};
  int li = 0, ls = 0, lb = 0, issued = 0;
  __amdgpu_buffer_rsrc_t xbuf = buffer(p.x, 0), wbuf = xbuf, xsbuf = xbuf, wsbuf = xbuf;
  const uint8_t *xsrc = nullptr, *wsrc = nullptr;
  uint32_t odd = 0;
  auto seek = [&] {
    ls = 0;
    for (; li < count; ++li) {
      lt = narrow_tile(sm, li);
      if (lt.steps > 0) break;
    }
    if (li >= count) return;
    if constexpr (TG) {
      xsrc = p.x + 128 * (lt.blk0 * p.K + lt.row0);
      wsrc = p.w + 128 * (lt.blk0 * p.N + lt.col0);
    } else {
      const uint32_t K = static_cast<uint32_t>(p.K), lds = static_cast<uint32_t>(p.lds);
      const uint32_t cols = static_cast<uint32_t>(min(static_cast<int>(p.N) - lt.col0, kNarrow));
      xbuf = buffer(p.x + static_cast<int64_t>(lt.row0) * p.ldx, (lt.rows - 1) * static_cast<uint32_t>(p.ldx) + K);
      wbuf = buffer(p.w + (static_cast<int64_t>(lt.g) * p.N + lt.col0) * p.K, cols * K);
      xsbuf = buffer(p.xs + lt.row0 * p.lds, lt.rows * lds);
      const int size = KIND == kGmmF32 ? 4 : 1;
      const uint8_t* src = static_cast<const uint8_t*>(p.ws) + (static_cast<int64_t>(lt.g) * lt.steps * nb + lt.col0 / 128) * size;
      odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src)) & 3;
      wsbuf = buffer(src - odd, (static_cast<uint32_t>(lt.steps * nb * size) + odd + 3) & ~3u);
    }
  };
  const int lr = 8 * wave + (lane >> 3);         // the staged row that the lane fills
  const uint32_t ldx = TG ? 128u : static_cast<uint32_t>(p.ldx), ldw = TG ? 128u : static_cast<uint32_t>(p.K);
  const uint32_t xc = 16 * ((lane & 7) ^ swz_run(lr)), wch = 16 * ((lane & 7) ^ (OUT_BF16 ? swz_quads(lr) : swz_run(lr)));
  // one load of each operand a wave; waves 0 and 1 bring the scales as well
  auto load = [&] {
    uint32_t xo = lr * ldx + xc, wo = lr * ldw + wch;
    if (!TG && 128 * ls + 128 > p.K) {
      const uint32_t end = static_cast<uint32_t>(p.K) - 128u * ls;
      xo = xc < end ? xo : kNowhere;
      wo = wch < end ? wo : kNowhere;
    }
    const uint32_t at = TG ? 0u : 128u * ls;
    if constexpr (TG) {
      xbuf = buffer(xsrc, 128u * lt.rows);
      wbuf = buffer(wsrc, 128u * static_cast<uint32_t>(min(static_cast<int>(p.N) - lt.col0, kNarrow)));
      xsrc += 128 * p.K;
      wsrc += 128 * p.N;
    }
    if (wave == 0) {
      if constexpr (TG) {
        const __amdgpu_buffer_rsrc_t b = buffer(p.xs + (static_cast<int64_t>(lt.blk0) + ls) * p.K + lt.row0, static_cast<uint32_t>(lt.rows));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)sm.xs[lb], 4, 4 * lane, 0, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xsbuf, (lds_void*)sm.xs[lb], 4, lane * static_cast<uint32_t>(p.lds), ls & ~3, 0, 0);
      }
    } else if (wave == 1) {
      if constexpr (TG) {
        const __amdgpu_buffer_rsrc_t b = buffer(static_cast<const uint8_t*>(p.ws) + (static_cast<int64_t>(lt.blk0) + ls) * p.N + lt.col0,
                                                static_cast<uint32_t>(min(static_cast<int>(p.N) - lt.col0, kNarrow)));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)sm.ws[lb], 4, 4 * lane, 0, 0, 0);
      } else {
        const uint32_t scale_at = KIND == kGmmF32 ? 4u * ls * nb : (odd + ls * nb) & ~3u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wsbuf, (lds_void*)sm.ws[lb], 4, scale_at, 0, 0, 0);
      }
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wbuf, (lds_void*)(sm.w[lb] + 1024 * wave), 16, wo, at, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_void*)(sm.x[lb] + 1024 * wave), 16, xo, at, 0, 0);
    order();
    lb = lb + 1 == NST ? 0 : lb + 1;
    ++issued;
    if (++ls == lt.steps) {
      ++li;
      seek();
    }
  };
  seek();
#pragma unroll
  for (int j = 0; j < NST - 1; ++j)
    if (li < count) load();
  const int wrow = 32 * wc + frag_col<OUT_BF16>(0, l15);
  const uint32_t xa0 = lds_addr(sm.x[0]) + (16 * wr + l15) * 128 + 16 * (grp ^ swz_run(l15));
  const uint32_t wa0 = lds_addr(sm.w[0]) + wrow * 128 + 16 * (grp ^ (OUT_BF16 ? swz_quads(wrow) : swz_run(wrow)));
  int done = 0, b = 0;
#pragma clang loop unroll(disable)
  for (int i = 0; i < count; ++i) {
    const WideTile t = narrow_tile(sm, i);
    v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
#pragma clang loop unroll(disable)
    for (int s = 0; s < t.steps; ++s) {
      // the stage is there when at most the six behind it are outstanding (and what was stored before them)
      if (issued - done < NST - 1)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      else if (wave < 2)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(3 * (NST - 2)));
      else
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * (NST - 2)));
      step_barrier();                            // every wave's loads are; the stage before is read
      if (li < count) load();
      ++done;
      if (16 * wr < t.rows) {
        const uint32_t xa = xa0 + b * static_cast<uint32_t>(sizeof(sm.x[0])), wa = wa0 + b * static_cast<uint32_t>(sizeof(sm.w[0]));
        const v8i x = frag(__builtin_bit_cast(uint4, lds_read<v4i>(xa)), __builtin_bit_cast(uint4, lds_read<v4i>(xa ^ 64u)));
        const uint32_t xsa = lds_addr(sm.xs[0]) + b * static_cast<uint32_t>(sizeof(sm.xs[0])), wsa = lds_addr(sm.ws[0]) + b * static_cast<uint32_t>(sizeof(sm.ws[0]));
        uint32_t xs, ws[2];
        float factor = 1.0f;
        if constexpr (TG) {
          xs = lds_read<uint8_t>(xsa + 16 * wr + l15);
#pragma unroll
          for (int f = 0; f < 2; ++f) ws[f] = lds_read<uint8_t>(wsa + wrow + frag_col<OUT_BF16>(f, 0));
        } else {
          xs = lds_read<uint32_t>(xsa + 4 * (16 * wr + l15)) >> (8 * (s & 3));
          if constexpr (KIND == kGmmF32) {
            const F32Scale sc = split_scale(lds_read<uint32_t>(wsa));
            factor = sc.factor;
            xs = lowered(xs & 255u, sc.down);
            ws[0] = ws[1] = sc.code;
          } else {
            const uint32_t byte = (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.ws)) + (static_cast<uint32_t>(t.g) * t.steps + s) * nb + t.col0 / 128) & 3;
            ws[0] = ws[1] = lds_read<uint8_t>(wsa + byte);
          }
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint32_t at = frag_col<OUT_BF16>(f, 0) * 128;
          const v8i w = frag(__builtin_bit_cast(uint4, lds_read<v4i>(wa + at)), __builtin_bit_cast(uint4, lds_read<v4i>((wa ^ 64u) + at)));
          if constexpr (KIND == kGmmF32)
            acc[f] += factor * mfma_scaled(w, ws[f], x, xs, v4f{0.f, 0.f, 0.f, 0.f});
          else
            acc[f] = mfma_scaled(w, ws[f], x, xs, acc[f]);
        }
      }
      b = b + 1 == NST ? 0 : b + 1;
    }
    if (16 * wr + l15 < t.rows) {
      const int64_t row = (TG ? t.g * p.K + t.row0 : t.row0) + 16 * wr + l15;
      if (OUT_BF16) {
        const int64_t c = t.col0 + 32 * wc + 8 * grp;
        if (c < p.N)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.N + c) =
              make_uint4(pack_bf16(acc[0][0], acc[0][1]), pack_bf16(acc[0][2], acc[0][3]), pack_bf16(acc[1][0], acc[1][1]), pack_bf16(acc[1][2], acc[1][3]));
      } else {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int64_t c = t.col0 + 32 * wc + 16 * f + 4 * grp;
          if (c < p.N) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * p.N + c) = make_float4(acc[f][0], acc[f][1], acc[f][2], acc[f][3]);
        }
      }
    }
  }
  if constexpr (!TG) zero_rows<OUT_BF16, kWideThreads>(p, n_rows);
}

template <Kind KIND, bool OUT_BF16, int MI>
void launch_few(const B128Args& p, hipStream_t st) {
  const int64_t tiles = b128::few_tiles(p.El, p.M, 16 * MI);
  b128_few_kernel<KIND, OUT_BF16, MI><<<static_cast<unsigned>(tiles * (p.N / 16)), 64 * kSplit, 0, st>>>(p, static_cast<int>(tiles));
}

template <Kind KIND, bool OUT_BF16>
hipError_t launch_b128(const B128Args& p, hipStream_t st) {
  const b128::Choice c = KIND == kTgmm ? b128::gradient_kernel(p.El, p.K, p.N, num_cus()) : b128::product_kernel(p.El, p.M, p.N, num_cus());
  if (c == b128::kWideTiles) {
    b128_wide_kernel<KIND, OUT_BF16><<<num_cus(), kWideThreads, 0, st>>>(p);
  } else if (c == b128::kNarrowTiles) {
    b128_narrow_kernel<KIND, OUT_BF16><<<num_cus(), kWideThreads, 0, st>>>(p);
  } else if constexpr (KIND != kTgmm) {
    if (c == b128::kFew64) launch_few<KIND, OUT_BF16, 4>(p, st);
    else if (c == b128::kFew32) launch_few<KIND, OUT_BF16, 2>(p, st);
    else launch_few<KIND, OUT_BF16, 1>(p, st);
  }
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
  // row offsets inside a tile, and a group's weights' scales, are 32-bit; a tile's rows span less than 2^31 bytes, so that
  // chunks past K, at 2^31, lie outside its buffer
  if (M > INT32_MAX - 1 || K > moe::kMaxLength || ldl > moe::kMaxLength || N > moe::kMaxLength || N * moe_cdiv(K, 128) > INT32_MAX) return MOE_ERR_SHAPE;
  // the tile table of any split of M rows into the groups stays below 2^31 entries
  if ((moe_cdiv(M, 16) + num_local_experts + 1) * (N / 16) > INT32_MAX) return MOE_ERR_SHAPE;
  if (ldl < K || ldl % 16 || lds < moe_cdiv(K, 128) || lds % 16 || lds > moe::kMaxScaleStride) return MOE_ERR_SHAPE;
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
  if (M < 0 || K <= 0 || N <= 0 || K % 16 || N % 16 || K > moe::kMaxLength || N > moe::kMaxLength) return MOE_ERR_SHAPE;
  if (E <= 0 || E > 1024 || group_offset < 0 || num_local_experts < 0 || num_local_experts > kMaxLocal ||
      group_offset > E - num_local_experts)
    return MOE_ERR_SHAPE;
  if (M > (int64_t{1} << 23) || M + 128 * static_cast<int64_t>(E) > (int64_t{1} << 23)) return MOE_ERR_SHAPE;
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
  const moe::B128Args p{lhs_t, 0, lhs_scale, 0, rhs_t, rhs_scale, group_sizes, group_offset, num_local_experts, M, K, N, out,
                        static_cast<int32_t*>(ws)};
  const hipError_t e = out_dtype == MOE_BF16 ? moe::launch_b128<moe::kTgmm, true>(p, st) : moe::launch_b128<moe::kTgmm, false>(p, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
