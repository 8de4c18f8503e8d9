/*
 * moe_fp8.h -- C ABI of libmoefp8.so, the fp8 mixture-of-experts
 * grouped-matmul hot path for AMD Instinct MI355X (gfx950).
 *
 * The path, as the MaxText pull requests "Quantize activations before EP all
 * gather" (PR 4812), "Support quantization for tokamax gmm v2" (PR 4451) and
 * "Keep qwix out of tpu-inference's fused MoE kernel and pre-quantize
 * weights" (PR 5136) describe it:
 *   1. per-token absmax quantization of activations to float8_e4m3fn;
 *   2. a stable ragged sort of the routed rows into contiguous per-expert
 *      groups (group_sizes, group_offset), moving fp8 rows and their scales;
 *   3. the grouped matmul of fp8 operands with a 32-bit accumulator, a per-row
 *      lhs scale and per-channel or blockwise [E, blocks, 1, N] rhs scales
 *      (gmm), and its transposed form for weight gradients (tgmm);
 *   4. the un-sort plus top-k weighted gather-reduce back to token rows.
 *
 * Conventions shared by every call
 *   - Every tensor argument is caller-owned DEVICE memory, row-major and
 *     densely packed, unless a comment says "host".  The library allocates
 *     nothing, frees nothing and never synchronises (except
 *     moe_debug_check).  Scratch memory comes from the caller's workspace
 *     `ws` of `ws_bytes` bytes, sized by moe_workspace_bytes().  The first
 *     int32 of a workspace is a sticky device-error word: the caller zeroes a
 *     workspace once before its first use; kernels OR error bits into it
 *     (MOE_DEVERR_*) and never clear it.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL is the default
 *     stream).  The return value reports host-side validation and launch
 *     errors only; data-dependent problems (an expert id out of range, a
 *     negative group size, more local rows than the buffer holds) set the
 *     sticky error word, kernels clamp so that no access leaves its buffer,
 *     and the affected outputs are unspecified.
 *   - Unsupported combinations are rejected with MOE_ERR_UNSUPPORTED, never
 *     silently ignored.  Zero-sized problems return MOE_OK after writing
 *     whatever outputs are defined for them (zeros).
 *   - Element types: bf16 = bfloat16 bit patterns (uint16), f32 = IEEE
 *     binary32, e4m3fn = OCP float8 E4M3 (bias 7, max 448, no infinities,
 *     NaN = S.1111.111; not the "fnuz" variant).
 *   - Calls are stateless and may be issued from several host threads.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define MOE_OK 0
#define MOE_ERR_NULL 1          /* a required pointer is NULL */
#define MOE_ERR_SHAPE 2         /* sizes inconsistent or outside the supported range */
#define MOE_ERR_UNSUPPORTED 3   /* a valid but unsupported combination */
#define MOE_ERR_WORKSPACE 4     /* workspace missing or too small */
#define MOE_ERR_HIP 5           /* a HIP launch failed */

/* element types */
#define MOE_DTYPE_DEFAULT (-1)
#define MOE_BF16 0
#define MOE_F32 1
#define MOE_E4M3FN 2
#define MOE_MX4 3               /* microscaled 4-bit: see moe_quantize_rows_mx4 */
#define MOE_E8M0 4              /* scale bytes s that stand for 2^(s - 127), 255 for NaN */

/* activation-scale granularity */
#define MOE_SCALE_ROW_DYNAMIC 0     /* one scale per row, from the row's absmax: [R] */
#define MOE_SCALE_TENSOR_DYNAMIC 1  /* one scale from the whole tensor's absmax: [1] */
#define MOE_SCALE_TENSOR_STATIC 2   /* one fixed scale given by the caller: [1] */
#define MOE_SCALE_TENSOR_FROM_ROW_AMAX 3 /* one scale from caller-given row maxima: [1] */

/* activation applied before quantization */
#define MOE_ACT_NONE 0
#define MOE_ACT_SILU_MUL 1          /* quantize silu(x) * x_up (gated FFN) */

/* router scores */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

/* operation ids for moe_workspace_bytes */
#define MOE_OP_QUANTIZE_ROWS 0
#define MOE_OP_SORT_BY_EXPERT 1
#define MOE_OP_GMM 2
#define MOE_OP_TGMM 3
#define MOE_OP_GATHER_REDUCE 4
#define MOE_OP_QUANTIZE_WEIGHTS 5
#define MOE_OP_GMM_MX4 6
#define MOE_OP_FFN_TOKENS 7
#define MOE_OP_GMM_B128 8
#define MOE_OP_TGMM_B128 9
#define MOE_OP_BALANCE 10

/* bits of the sticky device-error word (first int32 of a workspace) */
#define MOE_DEVERR_EXPERT_ID 1      /* an expert id outside [0, E) */
#define MOE_DEVERR_GROUP_SIZE 2     /* a negative group size */
#define MOE_DEVERR_ROWS 4           /* local rows exceed the row capacity */
#define MOE_DEVERR_SEQUENCE 8       /* sequence offsets that decrease or leave the rows */

/*
 * moe_quantize_rows -- absmax quantization of activations to e4m3fn.
 * Defined by "Quantize activations before EP all gather" (description: the
 * activations are quantized before the expert-parallel all-gather and the
 * activation sort; review comments on ragged_sort.py: a per-token scale has
 * the token dimension first) and by the schemes of "Support quantization
 * for tokamax gmm v2" (fp8_dynamic = absmax, fp8_static_wa = fixed scale).
 *
 *   x        [R, C] bf16.  With act == MOE_ACT_SILU_MUL, x is the gate a and
 *            x_up [R, C] bf16 the up projection b, and the quantized matrix is
 *            h = f32(silu(a) * b), silu(a) = f32(a / f32(1 + exp(-a))), using
 *            the library's pinned float32 exp (Cody-Waite reduction, degree-7
 *            Taylor polynomial, no fused multiply-add).  x_up must be NULL
 *            otherwise.
 *   scale_mode, static_scale: see MOE_SCALE_*; static_scale must be a
 *            positive finite float for MOE_SCALE_TENSOR_STATIC.
 *   q        [R, C] e4m3fn out.  q = e4m3(clip(f32(v / s), -448, 448)) with an
 *            IEEE float32 divide and round-to-nearest-even (sign kept,
 *            subnormals kept).
 *   scale    out: [R] f32 (row mode) or [1] f32 (tensor modes);
 *            s = f32(amax / 448), or 1.0 when amax is 0.
 *   row_amax optional [R] f32 out (may be NULL): each row's absmax.  With
 *            MOE_SCALE_TENSOR_FROM_ROW_AMAX it is an INPUT instead (required):
 *            the rows' absmax as an earlier row-mode call on the same rows
 *            wrote it; the scale is then f32(max(row_amax) / 448) (1.0 when
 *            that is 0), which equals MOE_SCALE_TENSOR_DYNAMIC's result
 *            without its absmax pass over x.
 *   ws       needed only for MOE_SCALE_TENSOR_DYNAMIC (may be NULL otherwise).
 * R >= 0; C > 0 and a multiple of 16.  Inputs must be finite.
 */
int moe_quantize_rows(const void* x, const void* x_up, int act, int64_t R, int64_t C,
                      int scale_mode, float static_scale, uint8_t* q, float* scale,
                      float* row_amax, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_quantize_rows_strided -- moe_quantize_rows over inputs whose rows are
 * ldx elements apart (the same step, "Support quantization for tokamax gmm
 * v2" absmax scheme; for the gated FFN, the requantization of silu(a) * b
 * where a and b are the two column halves of one grouped-matmul output).
 *   ldx      row stride of x and x_up in elements; ldx >= C, a multiple of 8,
 *            and x, x_up 16-byte aligned (MOE_ERR_SHAPE otherwise).  q stays
 *            [R, C] contiguous.  Every other argument, the result and the
 *            errors are those of moe_quantize_rows, which is this call with
 *            ldx = C.
 */
int moe_quantize_rows_strided(const void* x, const void* x_up, int64_t ldx, int act, int64_t R, int64_t C,
                              int scale_mode, float static_scale, uint8_t* q, float* scale,
                              float* row_amax, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_quantize_weights -- offline blockwise absmax quantization of expert
 * weights, the pre-quantization of "Keep qwix out of tpu-inference's fused
 * MoE kernel and pre-quantize weights" ("Changes in this PR": float8_e4m3fn
 * weights with [E, blocks, 1, N] scales, blockwise or channelwise).
 *
 *   w        [E, K, N] bf16 (contraction dim K, output channels N).
 *   kb, nb   scale blocks: block (b, c) covers K rows b*K/kb.. and columns
 *            c*N/nb..; kb divides K, nb divides N.  kb = 1, nb = N is
 *            per-output-channel.
 *   scale_mode MOE_SCALE_ROW_DYNAMIC (absmax of each block) or
 *            MOE_SCALE_TENSOR_STATIC (every block gets static_scale).
 *   transpose_out 0: q is [E, K, N]; 1: q is [E, N, K] (contraction dim
 *            contiguous, the layout moe_gmm_fp8 reads with transpose_rhs = 1).
 *   q        e4m3fn out; scale [E, kb, 1, nb] f32 out (s = f32(amax/448), 1.0
 *            for an all-zero block), q = e4m3(clip(f32(w / s), -448, 448)).
 * K, N multiples of 16.  Setup-time call; needs no workspace.
 */
int moe_quantize_weights(const void* w, int64_t E, int64_t K, int64_t N, int32_t kb, int32_t nb,
                         int scale_mode, float static_scale, int transpose_out, uint8_t* q,
                         float* scale, void* stream);

/*
 * moe_quantize_rows_i8 -- absmax quantization of activations to symmetric
 * int8 codes, the activation side of the int8 variant: "Keep qwix out of
 * tpu-inference's fused MoE kernel and pre-quantize weights" ("Changes in
 * this PR") allows int8 weights beside e4m3fn ones, and no matrix core
 * multiplies int8 by fp8 codes, so int8 weights take int8 activations, with
 * the per-token scales of "Quantize activations before EP all gather".
 *
 *   x        [R, C] bf16, rows contiguous, 16-byte aligned; C a multiple
 *            of 16.
 *   scale_mode MOE_SCALE_ROW_DYNAMIC (scale [R]), MOE_SCALE_TENSOR_DYNAMIC
 *            (scale [1] from the whole tensor; row_amax [R] is required and
 *            receives the rows' maxima), MOE_SCALE_TENSOR_STATIC (scale[0] =
 *            static_scale, finite and > 0) or MOE_SCALE_TENSOR_FROM_ROW_AMAX
 *            (scale [1] from the caller's row_amax [R]).
 *   q        [R, C] int8 out, 8-byte aligned: q = clip(rint(f32(x / s)),
 *            -127, 127), ties to even; s = f32(amax / 127), 1.0 for an
 *            all-zero row or tensor.
 *   row_amax [R] f32, optional in row mode (the rows' absmax out).
 * Needs no workspace.  MOE_ERR_SHAPE for a bad size, alignment or static
 * scale, MOE_ERR_NULL for a missing buffer, MOE_ERR_UNSUPPORTED for an
 * unknown mode; R = 0 writes only the tensor scale.
 */
int moe_quantize_rows_i8(const void* x, int64_t R, int64_t C, int scale_mode, float static_scale, int8_t* q,
                         float* scale, float* row_amax, void* stream);

/*
 * moe_quantize_weights_i8 -- moe_quantize_weights with int8 codes (the same
 * passage allows int8 weights with the same [E, blocks, 1, N] scales):
 * s = f32(amax / 127) per block (1.0 for an all-zero block),
 * q = clip(rint(f32(w / s)), -127, 127) with ties to even.  Arguments,
 * layouts and errors as in moe_quantize_weights; q is int8.
 */
int moe_quantize_weights_i8(const void* w, int64_t E, int64_t K, int64_t N, int32_t kb, int32_t nb,
                            int scale_mode, float static_scale, int transpose_out, int8_t* q,
                            float* scale, void* stream);

/*
 * moe_sort_by_expert -- stable ragged sort of routed rows into per-expert
 * groups, and the gather of the quantized token rows into that order.
 * Defined by "Quantize activations before EP all gather" (review comments on
 * ragged_sort.py: qvalue rows are gathered by the sorted token indices into
 * this shard's window of sorted rows; the scale is gathered with them only
 * when it is per token, a per-tensor scale passes through).
 *
 *   expert_ids [T, k] int32: routed expert of slot j of token t; the flat
 *            routed index is f = t*k + j.
 *   E        number of experts (1 <= E <= 1024); group_offset, num_local_experts:
 *            this GPU's experts are [group_offset, group_offset + num_local_experts).
 *   perm     [T*k] int32 out: flat index f of each globally sorted row; the
 *            sort is stable (equal expert ids keep increasing f).
 *   inv_pos  [T*k] int32 out: local sorted row of f, or -1 when f routes to a
 *            non-local expert.  Local sorted row 0 is the first row of expert
 *            group_offset (compact window).
 *   group_sizes [E] int32 out: rows per expert (global histogram).
 *   xq       optional [T, H] e4m3fn token rows (NULL skips the row gather);
 *   xscale   their scale: [T] f32 when xscale_mode == MOE_SCALE_ROW_DYNAMIC,
 *            otherwise [1] and passed through (ss may then be NULL).
 *   xs       [M_cap, H] e4m3fn out: xs[r] = xq[perm[start + r] / k] for the n
 *            local rows, zero for rows [n, M_cap).
 *   ss       [M_cap] f32 out (row mode): the gathered scales, zero past n.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_SORT_BY_EXPERT, T*k, 0, 0, E).
 * Invalid expert ids set MOE_DEVERR_EXPERT_ID and are sorted after every
 * valid row without entering any group; n > M_cap sets MOE_DEVERR_ROWS and
 * rows past M_cap are dropped.  H is a multiple of 16 (when xq is given).
 */
int moe_sort_by_expert(const int32_t* expert_ids, int64_t T, int32_t k, int32_t E,
                       int32_t group_offset, int32_t num_local_experts, const uint8_t* xq,
                       const float* xscale, int xscale_mode, int64_t H, int64_t M_cap,
                       int32_t* perm, int32_t* inv_pos, int32_t* group_sizes, uint8_t* xs,
                       float* ss, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_sort_gather_rows -- the row gather of moe_sort_by_expert alone, on the
 * metadata an earlier moe_sort_by_expert call (with xq NULL) wrote: its
 * inv_pos and the window header in its workspace ws.  The same bytes as the
 * one-call sort; lets the metadata run while the token rows are still being
 * quantized ("Quantize activations before EP all gather": the sort's order
 * depends on the routing only, the gathered rows on the quantized tokens).
 *   xq, xscale, xscale_mode, H, M_cap, xs, ss: as in moe_sort_by_expert.
 *   inv_pos  [T*k] from that call; ws: that call's workspace, unchanged
 *            since (the call must be ordered before this one on the device).
 * Errors: MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_NULL, MOE_ERR_WORKSPACE.
 */
int moe_sort_gather_rows(const uint8_t* xq, const float* xscale, int xscale_mode, const int32_t* inv_pos,
                         int64_t T, int32_t k, int64_t H, int64_t M_cap, uint8_t* xs, float* ss, void* ws,
                         size_t ws_bytes, void* stream);

/* Bytes of the device array that moe_sort_by_expert_noalloc uses in place of
 * a workspace (one per GPU). */
#define MOE_SORT_NOALLOC_SCRATCH_BYTES (2u << 20)

/*
 * moe_sort_by_expert_noalloc -- moe_sort_by_expert that allocates nothing and
 * takes no workspace, for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid it.
 * The sort's scratch (the window header and the per-tile histogram table)
 * lives in a library-owned device array of MOE_SORT_NOALLOC_SCRATCH_BYTES
 * bytes, one per GPU, held from the first call on that GPU until the process
 * ends.  Every call on a GPU shares that GPU's array: calls that overlap on
 * one GPU (different streams, or several host threads) race and must be
 * ordered by the caller.
 *   device_error  optional [1] int32 device out (may be NULL, then dropped):
 *            the MOE_DEVERR_* bits of this call's device-data errors are
 *            OR'ed into it; the caller zeroes it.
 * Every other argument, the results and the errors are those of
 * moe_sort_by_expert.  Sizes whose workspace
 * (moe_workspace_bytes(MOE_OP_SORT_BY_EXPERT, T*k, 0, 0, E)) exceeds
 * MOE_SORT_NOALLOC_SCRATCH_BYTES return MOE_ERR_WORKSPACE before any launch:
 * T*k may be at most 4128768 with E = 64, 1043968 with E = 256 and 261632
 * with E = 1024.
 * No hipMalloc, hipFree or allocating call is made.
 */
int moe_sort_by_expert_noalloc(const int32_t* expert_ids, int64_t T, int32_t k, int32_t E,
                               int32_t group_offset, int32_t num_local_experts, const uint8_t* xq,
                               const float* xscale, int xscale_mode, int64_t H, int64_t M_cap,
                               int32_t* perm, int32_t* inv_pos, int32_t* group_sizes, uint8_t* xs,
                               float* ss, int32_t* device_error, void* stream);

/*
 * moe_quantize_sort_by_expert -- moe_quantize_rows followed by
 * moe_sort_by_expert in one pass over the activations, for the single-GPU
 * path where no all-gather sits between them (the quantized activation
 * sort of "Quantize activations before EP all gather"; the same per-token
 * absmax scheme of "Support quantization for tokamax gmm v2").  Each token's
 * bf16 row is read once and its e4m3fn codes go straight to its local
 * destination rows; a token with none is not quantized (unless `scale` asks
 * for its scale).
 *   x        [T, H] bf16, 16-byte aligned; H > 0, a multiple of 16.
 *   scale_mode MOE_SCALE_ROW_DYNAMIC, MOE_SCALE_TENSOR_STATIC (with
 *            static_scale as in moe_quantize_rows) or
 *            MOE_SCALE_TENSOR_FROM_ROW_AMAX (the tensor scale from the token
 *            maxima in row_amax, as in moe_quantize_rows);
 *            MOE_SCALE_TENSOR_DYNAMIC needs the whole tensor before any code
 *            and is MOE_ERR_UNSUPPORTED.
 *   expert_ids .. group_sizes, M_cap, ws, ws_bytes: as in moe_sort_by_expert
 *            (workspace of moe_workspace_bytes(MOE_OP_SORT_BY_EXPERT, ...)).
 *   xs       [M_cap, H] e4m3fn out: the bytes moe_quantize_rows then
 *            moe_sort_by_expert would write (rows [n, M_cap) zero).
 *   ss       row mode: [M_cap] f32 out, each local row's token scale (0 past
 *            n); static mode: unused, may be NULL.
 *   scale    optional: row mode [T] f32 out, every token's scale (then every
 *            token is quantized); static mode [1] f32 out = static_scale;
 *            required in MOE_SCALE_TENSOR_FROM_ROW_AMAX mode, [1] f32 out.
 *   row_amax row mode: optional [T] f32 out, every token's absmax (then every
 *            token is quantized); MOE_SCALE_TENSOR_FROM_ROW_AMAX: required
 *            [T] f32 input, the tokens' absmax as a row-mode pass wrote it;
 *            ignored in static mode.
 * Errors as in moe_sort_by_expert; device-data errors (bad expert ids, more
 * local rows than M_cap) set the same workspace error bits.
 */
int moe_quantize_sort_by_expert(const void* x, int64_t T, int64_t H, int scale_mode, float static_scale,
                                const int32_t* expert_ids, int32_t k, int32_t E, int32_t group_offset,
                                int32_t num_local_experts, int64_t M_cap, int32_t* perm, int32_t* inv_pos,
                                int32_t* group_sizes, uint8_t* xs, float* ss, float* scale, float* row_amax,
                                void* ws, size_t ws_bytes, void* stream);

/*
 * moe_gmm_fp8 -- grouped matmul of fp8 operands, the gmm_v2 call of "Quantize
 * activations before EP all gather" (review comment on the prequantized test:
 * lhs_q, rhs_q, group_sizes, rhs_scale, group_offset, no lhs quantization in
 * the kernel), with the 32-bit accumulator that "Keep qwix out of
 * tpu-inference's fused MoE kernel" shows fp8 x fp8 needs, and the
 * [E, blocks, 1, N] weight scales of its "Changes in this PR".
 *
 * For local group g (rows [o_g, o_g + m_g) of lhs, o_g = sum of
 * group_sizes[group_offset .. group_offset+g-1], m_g = group_sizes[group_offset+g]):
 *   out[r, c] = ls[r] * sum_b rs[g, b, 0, c*Nb/N] * sum_{k in block b} lhs[r, k] * W_g[k, c]
 * accumulated in float32 by the fp8 matrix cores, the lhs scale applied in
 * float32 before the single rounding to out_dtype; rows [n, M) are zero.
 *
 *   lhs      [M, K] e4m3fn; lhs_scale [M] (MOE_SCALE_ROW_DYNAMIC) or [1]
 *            (either tensor mode) f32.
 *   rhs      [E_loc, K, N] e4m3fn (transpose_rhs = 0), or [E_loc, N, K]
 *            (transpose_rhs = 1: W_g = rhs[g]^T, e.g. the input gradient
 *            against the forward weight).
 *   rhs_scale [E_loc, Kb, 1, Nb] f32; K/Kb and N/Nb must be multiples of 128
 *            unless Kb == 1 (resp. Nb == 1 or Nb == N).
 *   group_sizes [E] int32 device; E, group_offset, num_local_experts as in
 *            moe_sort_by_expert.
 *   out      [M, N], out_dtype MOE_BF16 (default) or MOE_F32.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_GMM, M, K, N, E): the
 *            error word, one counter per tile of a split last round, and one
 *            float32 slot of 144 x 256 per workgroup (about 36 MiB on a
 *            256-CU GPU).  Zeroed once before its first use; the counters
 *            return to zero at the end of every call.  With it, when an XCD's
 *            share of tiles leaves a last round that fills few of its
 *            workgroups, each of those tiles is split along K over several
 *            workgroups and their float32 sums are added in a fixed order
 *            (int8 with one K block: int32 sums, added exactly).  Any smaller
 *            workspace of at least 256 bytes also works, without the split:
 *            the fp8 results may then differ in the last bits (another
 *            association of the same float32 sums); the same workspace size
 *            gives the same bits on every call.  Calls that share a workspace
 *            must not overlap (same stream, or ordered by events).
 * K and N multiples of 16 (MOE_ERR_SHAPE otherwise); multiples of 128 take
 * the tiled matrix-core kernels, other sizes a plainer edge kernel with the
 * same results.  M >= 0, 1 <= E <= 1024, num_local_experts <= 1024.
 */
int moe_gmm_fp8(const uint8_t* lhs, const float* lhs_scale, int lhs_scale_mode, const uint8_t* rhs,
                const float* rhs_scale, int32_t Kb, int32_t Nb, int transpose_rhs,
                const int32_t* group_sizes, int32_t E, int32_t group_offset,
                int32_t num_local_experts, int64_t M, int64_t K, int64_t N, int out_dtype,
                void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_gmm_i8 -- moe_gmm_fp8 with int8 operands (codes in [-127, 127] from
 * moe_quantize_rows_i8 / moe_quantize_weights_i8), the int8 weights of "Keep
 * qwix out of tpu-inference's fused MoE kernel and pre-quantize weights"
 * ("Changes in this PR") with the 32-bit accumulator its description shows
 * quantized operands need.  The products are summed exactly in int32 by the
 * int8 matrix cores (exact for K up to 2^17); with one K block the sum is
 * converted to float32 once, with several each block's exact sum is scaled
 * and added in float32:
 *   out[r, c] = ls[r] * sum_b rs[g, b, 0, c*Nb/N] * P_b[r, c],
 *   P_b = sum_{k in block b} lhs[r, k] * W_g[k, c] (an integer).
 * Arguments, layouts, workspace, size rules and errors as in moe_gmm_fp8;
 * K <= 2^17 (MOE_ERR_SHAPE beyond).
 */
int moe_gmm_i8(const int8_t* lhs, const float* lhs_scale, int lhs_scale_mode, const int8_t* rhs,
               const float* rhs_scale, int32_t Kb, int32_t Nb, int transpose_rhs,
               const int32_t* group_sizes, int32_t E, int32_t group_offset,
               int32_t num_local_experts, int64_t M, int64_t K, int64_t N, int out_dtype,
               void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_tgmm_fp8 -- transposed grouped matmul for weight gradients, the tgmm2
 * of "Support quantization for tokamax gmm v2" ("What this does": quantized
 * gmm2 / tgmm2, backward split into sub-functions):
 *   out[g, k, c] = (ls[k] * rs[c]) * sum_{r in group g} lhs[r, k] * rhs[r, c]
 * accumulated in float32; an empty local group gives zeros.
 *
 *   lhs      [M, K] e4m3fn with lhs_scale of lhs_scale_len 1 or K entries;
 *   rhs      [M, N] e4m3fn with rhs_scale of rhs_scale_len 1 or N entries.
 *            Scales must be constant along the contracted rows (a per-row
 *            scale does not factor out of the sum and is rejected).
 *   out      [E_loc, K, N], out_dtype MOE_F32 (default) or MOE_BF16.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_TGMM, M, K, N, E).
 * K and N multiples of 16 (MOE_ERR_SHAPE otherwise); multiples of 128 take
 * the tiled kernels, other sizes a plainer edge kernel with the same results.
 */
int moe_tgmm_fp8(const uint8_t* lhs, const float* lhs_scale, int32_t lhs_scale_len,
                 const uint8_t* rhs, const float* rhs_scale, int32_t rhs_scale_len,
                 const int32_t* group_sizes, int32_t E, int32_t group_offset,
                 int32_t num_local_experts, int64_t M, int64_t K, int64_t N, int out_dtype,
                 void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_tgmm_xt_cols -- columns (host out `cols`) of the transposed operand
 * layout that moe_sort_gather_transposed writes and moe_tgmm_fp8_xt reads,
 * for M local rows and E experts: 256 * ceil((M + 128 E) / 256).
 * MOE_ERR_SHAPE for M < 0 or E outside 1..1024.
 */
int moe_tgmm_xt_cols(int64_t M, int32_t E, int64_t* cols);

/*
 * moe_sort_gather_transposed -- the sort's row gather ("Quantize activations
 * before EP all gather": the fp8 token rows are gathered by the sorted token
 * indices into this shard's window) written straight into the layout the
 * weight-gradient product contracts over (tgmm2 of "Support quantization for
 * tokamax gmm v2"): the rows of each local group become a contraction axis
 * of their own.  For local group g with sorted rows rows_off[g] ..
 * rows_off[g] + m_g - 1 of the window and padded start P_g = 128 *
 * sum_{h<g} ceil(m_h / 128):
 *   xt[c, P_g + i] = code of x[perm[start + rows_off[g] + i] / k, c]   (i < m_g)
 *   xt[c, P_g + i] = 0                  (m_g <= i < 128 * ceil(m_g / 128))
 * with start = sum of group_sizes[0 .. group_offset-1] (the window's first
 * slot); columns past the last group's padded end are not written.
 *
 *   x        [T, H]: e4m3fn codes (x_dtype MOE_E4M3FN, e.g. from
 *            moe_quantize_rows with a tensor scale), or bf16 rows (MOE_BF16)
 *            quantized here with the static scale static_scale (> 0, finite)
 *            exactly as moe_quantize_rows(MOE_SCALE_TENSOR_STATIC) codes them.
 *   perm, group_sizes, E, group_offset, num_local_experts: as written by
 *            moe_sort_by_expert for the same routing (T*k slots, top-k = k).
 *   M        local rows of the weight-gradient call (rows of its dY).
 *   xt       [H, moe_tgmm_xt_cols(M, E)] bytes, row-major.
 *   scale_out optional device float [1]: receives static_scale (MOE_BF16).
 *   ws       workspace of at least 256 bytes (the error word).
 * H a multiple of 256 (MOE_ERR_UNSUPPORTED otherwise), 1 <= k <= 64.  A
 * source index outside the buffers is clamped (no access leaves them).
 * Errors: MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_NULL, MOE_ERR_WORKSPACE.
 */
int moe_sort_gather_transposed(const void* x, int x_dtype, float static_scale, int64_t T, int32_t k,
                               int64_t H, const int32_t* perm, const int32_t* group_sizes, int32_t E,
                               int32_t group_offset, int32_t num_local_experts, int64_t M, uint8_t* xt,
                               float* scale_out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_tgmm_fp8_xt -- moe_tgmm_fp8 with its lhs already in the transposed
 * layout of moe_sort_gather_transposed: xt [K, moe_tgmm_xt_cols(M, E)]
 * (column P_g + i = row rows_off[g] + i of the sorted lhs, zeros in each
 * group's padding).  Same result as moe_tgmm_fp8 on the sorted rows, bit for
 * bit.  rhs [M, N] as there.  K a multiple of 256 and N of 128
 * (MOE_ERR_UNSUPPORTED otherwise).  ws: at least 256 + N * cols bytes
 * (moe_workspace_bytes(MOE_OP_TGMM, M, K, N, E) is enough).  Other arguments
 * and errors as in moe_tgmm_fp8.
 */
int moe_tgmm_fp8_xt(const uint8_t* xt, const float* lhs_scale, int32_t lhs_scale_len, const uint8_t* rhs,
                    const float* rhs_scale, int32_t rhs_scale_len, const int32_t* group_sizes, int32_t E,
                    int32_t group_offset, int32_t num_local_experts, int64_t M, int64_t K, int64_t N,
                    int out_dtype, void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_gather_reduce -- un-sort plus top-k weighted combine, the ragged
 * gather-reduce of "Quantize activations before EP all gather" (review
 * comments on ragged_gather_reduce_v2.py: rows are reduced over a valid-rows
 * mask; the output dtype is bf16 when unspecified or fp8):
 *   out[t, :] = sum_{j < k, inv_pos[t, j] >= 0} w[t, j] * y[inv_pos[t, j], :]
 * accumulated in float32 in slot order j = 0..k-1, one rounding at the end.
 *
 *   y        [rows, N], y_dtype MOE_BF16 or MOE_F32 (rows >= 1 + max inv_pos).
 *   inv_pos  [T, k] int32 (from moe_sort_by_expert); topk_weights [T, k] f32.
 *   out      [T, N]; out_dtype MOE_BF16 (also for MOE_DTYPE_DEFAULT and
 *            MOE_E4M3FN) or MOE_F32.
 * N a multiple of 8.  Needs no workspace.
 */
int moe_gather_reduce(const void* y, int y_dtype, const int32_t* inv_pos, const float* topk_weights,
                      int64_t T, int32_t k, int64_t N, int out_dtype, void* out, void* stream);

/*
 * moe_gather_reduce_backward -- the backward of moe_gather_reduce, for the
 * layer backward that "Support quantization for tokamax gmm v2" splits into
 * gmm / tgmm calls ("What this does"; its accuracy tables compare gradients
 * as well as outputs).  With out[t] = sum_j w[t, j] * y[inv_pos[t, j]]:
 *   dy[inv_pos[t, j], :] = bf16(w[t, j] * dout[t, :])   (one float32
 *                           product, rounded to nearest even)
 *   dw[t, j]             = sum_c dout[t, c] * y[inv_pos[t, j], c]  (float32)
 * for every slot whose inverse position is in [0, M_cap); other slots get
 * dw = 0.  Rows [n, M_cap) of dy are zero, n = sum of
 * group_sizes[group_offset .. group_offset + num_local_experts).
 *
 *   dout     [T, N] bf16, the gradient of the combined token rows.
 *   y        [M_cap, N] bf16, the expert outputs the forward combined.
 *   inv_pos  [T, k] int32 and group_sizes [E] int32, from moe_sort_by_expert
 *            (every local row is the image of exactly one slot).
 *   topk_weights [T, k] f32.
 *   dy       [M_cap, N] bf16 out; dw [T, k] f32 out.
 *   dy_q, dy_scale, dy_amax  optional (all NULL, or all set; N <= 8192):
 *            [M_cap, N] e4m3fn, [M_cap] f32, [M_cap] f32 out -- dy quantized
 *            per row exactly as moe_quantize_rows(dy, MOE_SCALE_ROW_DYNAMIC)
 *            would (codes, scales and row absmax), formed while the row is in
 *            registers instead of in a second pass over dy.
 * N a multiple of 8, k <= 64.  Needs no workspace.  Errors: MOE_ERR_SHAPE,
 * MOE_ERR_NULL, MOE_ERR_UNSUPPORTED (dy_q with N > 8192); T = 0 with
 * M_cap = 0 returns MOE_OK.
 */
int moe_gather_reduce_backward(const void* dout, const void* y, const int32_t* inv_pos,
                               const float* topk_weights, int64_t T, int32_t k, int64_t N,
                               const int32_t* group_sizes, int32_t E, int32_t group_offset,
                               int32_t num_local_experts, int64_t M_cap, void* dy, float* dw,
                               uint8_t* dy_q, float* dy_scale, float* dy_amax, void* stream);

/*
 * moe_silu_mul_backward -- gradients of the gated FFN's activation
 * h = silu(a) * b for an upstream gradient dh, the activation step of the
 * layer backward that "Support quantization for tokamax gmm v2" splits into
 * gmm / tgmm calls ("What this does").  A pinned float32 recipe, one
 * rounding per step, no fused multiply-add:
 *   den = 1 + e(-a) (the forward's pinned exp), s = 1 / den, q = a / den,
 *   db = dh * q,  da = (dh * b) * (s * (1 + a * (1 - s)))
 * each result rounded to bf16 (nearest even).
 *
 *   a, b     [R, C] bf16 with row stride lda elements (e.g. the two column
 *            halves of the fused input-projection output, lda = 2C).
 *   dh       [R, C] bf16, dense.
 *   da, db   [R, C] bf16 out with row stride ldo (e.g. the halves of one
 *            [R, 2C] buffer that the input-gradient gmm over [W0 | W1]^T
 *            reads as its lhs).
 * C, lda, ldo multiples of 8, lda >= C, ldo >= C.  Needs no workspace.
 * Errors: MOE_ERR_SHAPE, MOE_ERR_NULL; R = 0 returns MOE_OK.
 */
int moe_silu_mul_backward(const void* a, const void* b, int64_t lda, const void* dh, int64_t R, int64_t C,
                          void* da, void* db, int64_t ldo, void* stream);

/*
 * moe_router_topk -- the router in front of the sort: the k experts of every
 * token and their weights, from the token's logits z [E].
 *   scores   MOE_SCORE_SOFTMAX p_e = exp(z_e - m) / sum_f exp(z_f - m), or
 *            MOE_SCORE_SIGMOID p_e = 1 / (1 + exp(-z_e)), 0 for z_e below -700;
 *            renormalised weights are the ratios of such scores also where
 *            every chosen one is below float32's range
 *   choice   the k largest logits (scores rise with them), or with
 *            select_bias the k largest p_e + select_bias[e], formed in 64
 *            bits; in descending order, equal ones to the lower expert
 *   weights  weight_scale * p_e of the chosen; with renormalize
 *            weight_scale * p_e / (sum of the chosen p).  The bias enters the
 *            choice only.
 *
 *   logits   [T, E] bf16 or f32 (logits_dtype), rows ldl >= E elements apart.
 *            A logit of -inf (or NaN) takes the expert out for that token: it
 *            is chosen after every other one and has weight 0.  A row without
 *            any other logit (a padded token) gets experts 0 .. k-1 with
 *            weights 0, so that every id stays valid for the sort.  A logit
 *            of +inf is not supported (ids stay valid, weights unspecified).
 *   select_bias optional [E] f32, finite (NULL for none).
 *   expert_ids [T, k] int32 out; topk_weights [T, k] f32 out: what
 *            moe_sort_by_expert, moe_gather_reduce and moe_ffn_tokens take.
 * 1 <= E <= 1024, 1 <= k <= min(E, 64), weight_scale finite and > 0, T <=
 * 2^31.  Needs no workspace.  Errors: MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED
 * (type, score, renormalize not 0 or 1), MOE_ERR_NULL.
 */
int moe_router_topk(const void* logits, int logits_dtype, int64_t ldl, int64_t T, int32_t E, int32_t k, int score,
                    const float* select_bias, int renormalize, float weight_scale, int32_t* expert_ids,
                    float* topk_weights, void* stream);

/*
 * moe_router_topk_backward -- gradient of moe_router_topk's weights to the
 * logits, the choice held fixed.  dweights is what moe_gather_reduce_backward
 * writes as dw.  With g_j = weight_scale * dweights[t, j]:
 *   softmax                dz_e = p_e (g_e - sum_j g_j p_j), g_e = 0 unless chosen
 *   softmax, renormalize   dz_e = r_e (g_e - sum_j g_j r_j) for the chosen, 0
 *                          for the others; r = the softmax over the chosen
 *   sigmoid                dz_e = g_e p_e (1 - p_e)
 *   sigmoid, renormalize   the same with (g_e - sum_j g_j p_j / S) / S in
 *                          place of g_e, S = the chosen p's sum
 * Experts taken out by -inf, and every expert of a row without another
 * logit, get 0, and dweights of slots that hold such an expert take no part,
 * whatever they hold.
 *   logits .. weight_scale as in the forward call; expert_ids [T, k] as it
 *   wrote them (an id outside [0, E) takes no part; one given twice counts
 *   twice).
 *   dlogits  [T, E] out, logits_dtype, rows ldd >= E elements apart; must not
 *            overlap logits.
 * Sizes and errors as in moe_router_topk.
 */
int moe_router_topk_backward(const void* logits, int logits_dtype, int64_t ldl, const int32_t* expert_ids,
                             const float* dweights, int64_t T, int32_t E, int32_t k, int score, int renormalize,
                             float weight_scale, void* dlogits, int64_t ldd, void* stream);

/*
 * moe_quantize_rows_mx4 -- rows to the microscaled 4-bit format (the MXFP4
 * of the OCP Microscaling Formats specification): every 32 consecutive
 * elements share one e8m0 scale 2^(s - 127) and hold e2m1 codes (sign, two
 * exponent bits, one mantissa bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).
 *   scale    s = floor(log2(block absmax)) - 2 + 127, at least 0; 127 for a
 *            block of zeros; 255 (NaN) for a block with an element that is
 *            not finite: every element of it then reads back as NaN
 *   codes    v / scale (exact) to the nearest e2m1 value, ties to the even
 *            code, saturating at 6; the sign of zero is kept
 *   x, x_up, ldx, act  [R, C] bf16, rows ldx elements apart, as in
 *            moe_quantize_rows_strided (with MOE_ACT_SILU_MUL the matrix is
 *            silu(x) * x_up in float32 by the same recipe).
 *   q        [R, C/2] bytes out, rows ldq bytes apart: element 2i in the low
 *            half of byte i, 2i + 1 in the high half.
 *   scale    [R, C/32] bytes out, rows lds bytes apart.  q and scale may be
 *            parts of one row (scale = q + C/2, ldq = lds), which one gather
 *            then moves; bytes between the rows' parts are not written.
 * C a multiple of 32, ldx >= C and a multiple of 8, ldq >= C/2 and a multiple
 * of 16, lds >= C/32; x, x_up, q 16-byte aligned (MOE_ERR_SHAPE otherwise).
 * Expert weights stored [E, N, K] are rows too (R = E N, C = K).  Needs no
 * workspace.  Errors as in moe_quantize_rows_strided.
 */
int moe_quantize_rows_mx4(const void* x, const void* x_up, int64_t ldx, int act, int64_t R, int64_t C, uint8_t* q,
                          int64_t ldq, uint8_t* scale, int64_t lds, void* stream);

/*
 * moe_quantize_weights_mx4 -- expert weights w [E, K, N] bf16 to the 4-bit
 * format with blocks along the contraction K, stored contraction-contiguous:
 * q [E, N, K/2], scale [E, N, K/32] (the layout moe_gmm_mx4 and
 * moe_ffn_tokens read).  K a multiple of 32, N of 16; w and q 16-byte
 * aligned.  Setup-time call; needs no workspace.  Errors: MOE_ERR_SHAPE,
 * MOE_ERR_NULL; E = 0 returns MOE_OK.
 */
int moe_quantize_weights_mx4(const void* w, int64_t E, int64_t K, int64_t N, uint8_t* q, uint8_t* scale, void* stream);

/*
 * moe_dequantize_rows_mx4 -- the values of 4-bit rows, exactly.
 *   q, ldq, scale, lds as moe_quantize_rows_mx4 writes them; out [R, C] bf16
 *   (also for MOE_DTYPE_DEFAULT) or f32, rows ldo elements apart (ldo >= C, a
 *   multiple of 8), 16-byte aligned.  A block of scale code 255 reads as NaN.
 * Errors: MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_NULL.
 */
int moe_dequantize_rows_mx4(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds, int64_t R, int64_t C,
                            int out_dtype, void* out, int64_t ldo, void* stream);

/*
 * moe_gmm_mx4 -- moe_gmm_fp8 with 4-bit weights: for local group g (rows as
 * there)
 *   out[r, c] = ls[r] * sum_k X[r, k] * W_g[k, c]
 * accumulated in float32 by the scaled matrix cores, rounded once to
 * out_dtype; rows past the last local group's are zero.
 *   lhs      lhs_format MOE_E4M3FN: [M, K] e4m3fn, rows ldl bytes apart, with
 *            lhs_scale f32 [M] (MOE_SCALE_ROW_DYNAMIC) or [1] (the tensor
 *            modes) and lds = 0.
 *            lhs_format MOE_MX4: [M, K/2] codes, rows ldl bytes apart, and
 *            lhs_scale [M, K/32] e8m0 bytes, rows lds apart
 *            (moe_quantize_rows_mx4; lhs_scale_mode MOE_SCALE_ROW_DYNAMIC).
 *            Sorted rows of either kind come from moe_sort_by_expert /
 *            moe_sort_gather_rows, which move bytes.
 *   rhs      [E_loc, N, K/2] codes, rhs_scale [E_loc, N, K/32] e8m0 bytes
 *            (moe_quantize_weights_mx4).
 *   group_sizes .. num_local_experts, out, out_dtype as in moe_gmm_fp8.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_GMM_MX4, M, K, N, E).
 *            Scale rows of a 4-bit lhs that are not dword aligned (lds, or
 *            lhs_scale itself) are copied there first; calls that may overlap
 *            need a workspace each.
 * K a multiple of 32 and at most 2^22, N of 16, N * K / 32 below 2^31, ldl a
 * multiple of 16, at least a row's bytes and at most 2^23; lhs, rhs, rhs_scale,
 * out 16-byte aligned.  Errors as in moe_gmm_fp8.
 */
int moe_gmm_mx4(const uint8_t* lhs, int64_t ldl, const void* lhs_scale, int64_t lds, int lhs_format,
                int lhs_scale_mode, const uint8_t* rhs, const uint8_t* rhs_scale, const int32_t* group_sizes, int32_t E,
                int32_t group_offset, int32_t num_local_experts, int64_t M, int64_t K, int64_t N, int out_dtype,
                void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_ffn_tokens -- a whole gated expert layer for a few tokens (decoding):
 *   out[t, :] = sum_j w[t, j] * ((silu(x[t] W0_e) * (x[t] W1_e)) Wo_e), e = expert_ids[t, j]
 * over the slots whose expert is local, in slot order; a token without one
 * gets zeros.  The sorted path (quantize, sort, grouped matmuls, combine) is
 * for many tokens; here the rows are not sorted and nothing is quantized: the
 * activations stay bfloat16, sums and the hidden values 32-bit (the hidden
 * values enter the second product as two bfloat16 pieces), one rounding at
 * the end.  A token's result does not depend on the other tokens, neither on
 * their values nor on their experts: the same bits alone and in any batch.
 *   x        [T, H] bf16, rows ldx elements apart (a multiple of 8, 16-byte
 *            aligned); 0 <= T <= 64, T k <= 1024 (MOE_ERR_UNSUPPORTED beyond).
 *   expert_ids, topk_weights [T, k] int32 / f32, as moe_router_topk writes
 *            them; an id outside [0, E) sets MOE_DEVERR_EXPERT_ID and its
 *            slot takes no part; an expert given twice counts twice.
 *   E, group_offset, num_local_experts: as in moe_sort_by_expert.
 *   w_format MOE_E4M3FN: w01 [E_loc, 2I, H] (gate rows, then up rows), wo
 *            [E_loc, H, I] e4m3fn, contraction-contiguous, with f32 scales
 *            w01_scale [E_loc, kb01, 1, nb01] and wo_scale [E_loc, kbo, 1,
 *            nbo] under moe_gmm_fp8's rules; H and I multiples of 16.
 *            MOE_MX4: w01 [E_loc, 2I, H/2], wo [E_loc, H, I/2] codes, e8m0
 *            scales [E_loc, 2I, H/32] and [E_loc, H, I/32]; kb01 = nb01 = kbo
 *            = nbo = 0; H and I multiples of 32.  A scale of 255 (NaN)
 *            makes every result that its block enters NaN, whatever the codes.
 *            Scales of 253 and 254 are not supported (their values may pass
 *            bfloat16's range and become infinite; no quantizer here writes them).
 *   out      [T, H] bf16 (default) or f32.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_FFN_TOKENS, T*k, H, I, E),
 *            zeroed once before its first use (the error word).  Calls that
 *            share one must not overlap.
 * H, I <= 2^20.  w01, wo, out 16-byte aligned, the scales 4-byte.  Errors: MOE_ERR_SHAPE,
 * MOE_ERR_UNSUPPORTED, MOE_ERR_NULL, MOE_ERR_WORKSPACE.
 */
int moe_ffn_tokens(const void* x, int64_t ldx, const int32_t* expert_ids, const float* topk_weights, int64_t T, int32_t k,
                   int64_t H, int64_t I, int32_t E, int32_t group_offset, int32_t num_local_experts, int w_format,
                   const uint8_t* w01, const void* w01_scale, int32_t kb01, int32_t nb01, const uint8_t* wo,
                   const void* wo_scale, int32_t kbo, int32_t nbo, int out_dtype, void* out, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * moe_quantize_rows_b128 -- rows to e4m3fn with a scale for every block of
 * 128 elements (the last block of a row may be shorter): the format of the
 * b128 calls.
 *   scale    one e8m0 byte s a block, standing for 2^(s - 127): the smallest
 *            power of two with block absmax <= 448 * 2^(s - 127), at least
 *            2^-127; 127 for a block of zeros; 255 (NaN) for a block with an
 *            element that is not finite: every element of it, and every
 *            result of a product that it enters, is then NaN
 *   codes    v / scale (exact) to the nearest e4m3fn value, ties to even; the
 *            sign of zero is kept; 0 in a block of scale 255
 *   x, x_up, ldx, act  [R, C] bf16, rows ldx elements apart, as in
 *            moe_quantize_rows_strided (with MOE_ACT_SILU_MUL the matrix is
 *            silu(x) * x_up in float32 by the same recipe).
 *   q        [R, C] bytes out, rows ldq bytes apart.
 *   scale    [R, ceil(C / 128)] bytes out, rows lds bytes apart.  q and scale
 *            may be parts of one row (scale = q + C, ldq = lds), which one
 *            gather (moe_sort_by_expert, which moves bytes) then moves; bytes
 *            between the rows' parts are not written.
 * C a multiple of 16, ldx >= C and a multiple of 8, ldq >= C and a multiple
 * of 16, lds >= ceil(C / 128); x, x_up, q 16-byte aligned (MOE_ERR_SHAPE
 * otherwise).  Needs no workspace.  Errors as in moe_quantize_rows_strided.
 */
int moe_quantize_rows_b128(const void* x, const void* x_up, int64_t ldx, int act, int64_t R, int64_t C, uint8_t* q,
                           int64_t ldq, uint8_t* scale, int64_t lds, void* stream);

/*
 * moe_quantize_weights_b128 -- expert weights w [E, K, N] bf16 to e4m3fn with
 * an e8m0 scale (as in moe_quantize_rows_b128) for every block of 128 by 128,
 * in either or both orientations, in one pass:
 *   q, scale       [E, N, K] codes and [E, ceil(K/128), 1, ceil(N/128)] scales:
 *                  what moe_gmm_b128 reads for x W
 *   qt, scale_t    [E, K, N] codes and [E, ceil(N/128), 1, ceil(K/128)] scales:
 *                  what it reads for the input gradient dy W^T (contraction N)
 * The two hold the same values.  A pair may be NULL, not both pairs.
 * K and N multiples of 16; w, q, qt 16-byte aligned.  Needs no workspace.
 * Errors: MOE_ERR_SHAPE, MOE_ERR_NULL; E = 0 returns MOE_OK.
 */
int moe_quantize_weights_b128(const void* w, int64_t E, int64_t K, int64_t N, uint8_t* q, uint8_t* scale, uint8_t* qt,
                              uint8_t* scale_t, void* stream);

/*
 * moe_quantize_cols_b128 -- the rows of each local group to e4m3fn with a
 * scale for every 128 of its rows and column, every 128 rows laid out column
 * by column: the operand of the weight gradient, whose contraction runs along
 * a group's rows.  With the local groups' sorted rows rows_off[g] .. rows_off[g] + m_g - 1
 * and padded starts P_g = 128 * sum_{h<g} ceil(m_h / 128), as in
 * moe_sort_gather_transposed:
 *   qt[(P_g + i) / 128, c, i % 128]  code of V[rows_off[g] + i, c]   (i < m_g)
 *                                    0      (m_g <= i < 128 * ceil(m_g / 128))
 *   scale_t[P_g / 128 + b, c]        scale of rows 128 b .. of group g, column c
 * scales and codes formed as in moe_quantize_rows_b128 along those rows.
 * What lies past the last group's padded end, in both, is not written.
 *   V        the local sorted rows: with perm NULL, x itself, [M, C]; with
 *            perm [T*k] (moe_sort_by_expert's), V[r] = x[perm[start + r] / k],
 *            x [T, C] the tokens, start = sum of group_sizes[0 .. first_group-1].
 *   x, x_up, ldx, act as in moe_quantize_rows_b128.  T, k: as in the sort
 *            (k is 1 to 64); without perm T is x's row count, at least M.
 *   group_sizes, E, first_group, num_local_experts: as in the sort, whose
 *            group_offset is first_group here and in the products.
 *   M        local rows (rows of the weight gradient's operands).
 *   qt       [cols / 128, C, 128] bytes, scale_t [cols / 128, C] bytes, cols =
 *            moe_tgmm_xt_cols(M, E); both 16-byte aligned.
 *   ws       workspace of at least 256 bytes (the error word: negative sizes,
 *            more local rows than M; a row index outside x is clamped).
 * C a multiple of 16, M + 128 E <= 2^23.  Errors: MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED,
 * MOE_ERR_NULL, MOE_ERR_WORKSPACE.
 */
int moe_quantize_cols_b128(const void* x, const void* x_up, int64_t ldx, int act, int64_t T, int32_t k, const int32_t* perm,
                           const int32_t* group_sizes, int32_t E, int32_t first_group, int32_t num_local_experts,
                           int64_t M, int64_t C, uint8_t* qt, uint8_t* scale_t, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_gmm_b128 -- moe_gmm_fp8 with a scale for every block of 128 of both
 * operands: for local group g (rows as there)
 *   out[r, c] = sum_b sx[r, b] * sw[g, b, c / 128] * sum_{k in block b} X[r, k] * W_g[k, c]
 * accumulated in float32 by the scaled matrix cores, rounded once to
 * out_dtype; rows past the last local group's are zero.
 *   lhs      [M, K] e4m3fn, rows ldl bytes apart; lhs_scale [M, ceil(K/128)]
 *            e8m0 bytes, rows lds apart (moe_quantize_rows_b128).  Scale rows
 *            are read in whole pieces of 16 bytes, the last row's too.
 *   rhs      [E_loc, N, K] e4m3fn; rhs_scale [E_loc, ceil(K/128), 1,
 *            ceil(N/128)], of rhs_scale_dtype MOE_E8M0
 *            (moe_quantize_weights_b128) or MOE_F32 (any float32: weights as
 *            moe_quantize_weights or a checkpoint hold them in 128 x 128 blocks;
 *            a scale that is not finite is NaN, as 255 is; a block of scale 0
 *            adds nothing, but NaN where it holds or meets one).
 *   group_sizes .. num_local_experts, out, out_dtype as in moe_gmm_fp8.  One
 *            group (E = 1, its size M) is a plain linear layer.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_GMM_B128, M, K, N, E).
 * K and N multiples of 16 and at most 2^22, N * ceil(K/128) < 2^31; ldl a multiple
 * of 16, K to 2^22; lds a multiple of 16, at least ceil(K/128); lhs,
 * lhs_scale, rhs, out 16-byte aligned.  Errors as in moe_gmm_fp8.
 */
int moe_gmm_b128(const uint8_t* lhs, int64_t ldl, const uint8_t* lhs_scale, int64_t lds, const uint8_t* rhs,
                 const void* rhs_scale, int rhs_scale_dtype, const int32_t* group_sizes, int32_t E, int32_t first_group,
                 int32_t num_local_experts, int64_t M, int64_t K, int64_t N, int out_dtype, void* out, void* ws,
                 size_t ws_bytes, void* stream);

/*
 * moe_tgmm_b128 -- the weight gradient of moe_gmm_b128, both operands
 * quantized along the rows of each group (moe_quantize_cols_b128):
 *   out[g, k, c] = sum_b sx[b, k] * sy[b, c] * sum_{i < 128} lhs_t[b, k, i] * rhs_t[b, c, i]
 * over the blocks b of group g, accumulated in float32 by the scaled matrix
 * cores; an empty local group gives zeros.
 *   lhs_t    [cols / 128, K, 128] codes, lhs_scale [cols / 128, K]; rhs_t
 *            [cols / 128, N, 128], rhs_scale [cols / 128, N]; cols = moe_tgmm_xt_cols(M, E).
 *   group_sizes .. num_local_experts, M: as the operands were made with.
 *   out      [E_loc, K, N], out_dtype MOE_F32 (default) or MOE_BF16.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_TGMM_B128, M, K, N, E).
 * K and N multiples of 16 and at most 2^22, M + 128 E <= 2^23; all buffers 16-byte aligned.  Errors as
 * in moe_tgmm_fp8.
 */
int moe_tgmm_b128(const uint8_t* lhs_t, const uint8_t* lhs_scale, const uint8_t* rhs_t, const uint8_t* rhs_scale,
                  const int32_t* group_sizes, int32_t E, int32_t first_group, int32_t num_local_experts, int64_t M,
                  int64_t K, int64_t N, int out_dtype, void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_balance_loss -- the router's balance loss of every sequence of a batch,
 * and how often each expert was chosen.  With the shares p[t, e] of a token's
 * scores (MOE_SCORE_SOFTMAX: the softmax of its logits; MOE_SCORE_SIGMOID:
 * sigmoid(z_e) / sum_f sigmoid(z_f)), for sequence s of n tokens that have an
 * expert, c[e] choices of expert e:
 *   loss[s] = E / (k n^2) * sum_e c[e] * sum_t p[t, e]         (0 where n = 0)
 * which is 1 where either is even over the experts.  A share is held in float32,
 * off by a few units in its last place (0 below 2^-126 of the row's largest).
 *   logits, logits_dtype, ldl  [T, E] as in moe_router_topk.  A logit of -inf or
 *            NaN, or at or below -1e30 (a mask of the type's lowest value), takes
 *            its expert out for that token: no share, and no choice of it counts.
 *            A token whose every logit is out (a padded one) is no token here.
 *            +inf is not supported (its sequence's loss is unspecified).
 *   expert_ids [T, k] int32 as moe_router_topk wrote them (an id outside [0, E)
 *            does not count, one given twice counts twice).
 *   seq_offsets [S + 1] int32, device: sequence s is the tokens
 *            seq_offsets[s] .. seq_offsets[s+1] - 1 (it may be empty); rows
 *            outside all sequences take no part.  NULL with S = 1: all T rows.
 *            Offsets that decrease or leave [0, T] set MOE_DEVERR_SEQUENCE and
 *            are clamped; where they decrease, what the call writes for the
 *            sequences is unspecified.
 *   loss     [S] f32 out; counts [S, E] int32 out; tokens [S] int32 out: n.
 *   ws       workspace of moe_workspace_bytes(MOE_OP_BALANCE, T, S, 0, E).
 * The result's bits do not depend on the order in which the device runs.
 * 1 <= E <= 1024, 1 <= k <= min(E, 64), 0 <= T <= 2^31 - 1, 1 <= S <= 2^24.
 * Errors: MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_NULL, MOE_ERR_WORKSPACE.
 */
int moe_balance_loss(const void* logits, int logits_dtype, int64_t ldl, const int32_t* expert_ids, int64_t T, int32_t E,
                     int32_t k, int score, const int32_t* seq_offsets, int32_t S, float* loss, int32_t* counts,
                     int32_t* tokens, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_balance_loss_backward -- gradient of sum_s dloss[s] * loss[s] to the
 * logits, the choices held fixed:
 *   dz[t, e] = dloss[s] * E / (k n^2) * p_e * (c[e] - sum_f c[f] p_f) * r_e
 * r_e = 1 for softmax, 1 - sigmoid(z_e) for sigmoid scores; 0 for experts
 * taken out.
 *   logits .. S as in the forward call; counts, tokens as it wrote them (a
 *   data-parallel caller may have summed both over its ranks).
 *   dloss    [S] f32.
 *   accumulate 0: the rows of the sequences are written; 1: added, in float32,
 *            to what dlogits holds (the router's own gradient), rounded once.
 *   dlogits  [T, E], logits_dtype, rows ldd >= E elements apart; must not
 *            overlap logits.  Rows outside all sequences are left as they are.
 * Needs no workspace; offsets are clamped as in the forward call.
 */
int moe_balance_loss_backward(const void* logits, int logits_dtype, int64_t ldl, const int32_t* counts, const int32_t* tokens,
                              const float* dloss, int64_t T, int32_t E, int32_t k, int score, const int32_t* seq_offsets,
                              int32_t S, int accumulate, void* dlogits, int64_t ldd, void* stream);

/*
 * moe_workspace_bytes -- workspace size (host out `bytes`) for `op` with
 * problem sizes d0, d1, d2 and E:
 *   MOE_OP_QUANTIZE_ROWS   d0 = R, d1 = C, d2 = scale_mode
 *   MOE_OP_SORT_BY_EXPERT  d0 = T*k
 *   MOE_OP_GMM, MOE_OP_TGMM, MOE_OP_GMM_MX4, MOE_OP_GMM_B128,
 *   MOE_OP_TGMM_B128       d0 = M, d1 = K, d2 = N
 *   MOE_OP_FFN_TOKENS      d0 = T*k (at most 1024), d1 = H, d2 = I
 *   MOE_OP_BALANCE         d0 = T, d1 = S
 *   others                 only the error word
 * Every size is a multiple of 256 bytes and at least 256.
 */
int moe_workspace_bytes(int op, int64_t d0, int64_t d1, int64_t d2, int32_t E, size_t* bytes);

/*
 * moe_debug_check -- synchronises `stream` and copies the sticky error word
 * of workspace `ws` into host *device_error.  Debug use only.
 */
int moe_debug_check(const void* ws, void* stream, int32_t* device_error);

/* moe_status_string -- static text for a status code. */
const char* moe_status_string(int status);

/* moe_version -- library version as 10000*major + 100*minor + patch. */
int moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */
