"""Blocks of 128 e4m3fn elements that share one e8m0 scale: quantizers, the
grouped product and its weight gradient, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

"Keep qwix out of tpu-inference's fused MoE kernel and pre-quantize weights"
("Changes in this PR") gives the weights [E, blocks, 1, N] scales; here the
activations and the gradients have a scale for each block as well, and every
scale is a power of two.
"""

import numpy as np

from .codec import bf16_decode, e4m3_decode, e4m3_rne
from .quantize import silu_mul_f32

BLOCK = 128


def scale_codes(amax):
    """e8m0 codes for largest magnitudes: the smallest power of two, from
    2^-127 on, with amax <= 448 times it."""
    amax = np.asarray(amax, np.float64)
    fin = np.isfinite(amax)
    m, e = np.frexp(np.where(fin, amax, 1.0))              # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    code = np.maximum(np.where(m <= 0.875, e - 9, e - 8) + 127, 0)
    return np.where(~fin, 255, np.where(amax == 0, 127, code)).astype(np.uint8)


def scale_values(code):
    code = np.asarray(code)
    return np.where(code == 255, np.nan, np.ldexp(1.0, code.astype(np.int64) - 127))


def _codes(v, code):
    """Codes of float64 values with (broadcast) scale codes."""
    bad = code == 255
    y = np.where(bad, 0.0, v) / np.where(bad, 1.0, scale_values(np.where(bad, 127, code)))
    return np.where(bad, 0, e4m3_rne(y.astype(np.float32))).astype(np.uint8)       # (a power of two: the quotient is exact)


def _amax(b, axis):
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(b).all(axis=axis), np.abs(np.where(np.isfinite(b), b, 0)).max(axis=axis), np.inf)


def quantize_values(v):
    """Codes [R, C] and scale codes [R, ceil(C / 128)] of float64 rows."""
    v = np.asarray(v, np.float64)
    R, C = v.shape
    nb = -(-C // BLOCK)
    s = np.stack([scale_codes(_amax(v[:, b * BLOCK:(b + 1) * BLOCK], 1)) for b in range(nb)], axis=1)
    return _codes(v, np.repeat(s, BLOCK, axis=1)[:, :C]), s


def values(x_bits, x_up_bits=None):
    """float64 of bf16 rows (bits); with x_up the float32 silu(x) * x_up."""
    x = bf16_decode(x_bits)
    return np.asarray(x if x_up_bits is None else silu_mul_f32(x, bf16_decode(x_up_bits)), np.float64)


def quantize_rows_b128(x_bits, x_up_bits=None):
    return quantize_values(values(x_bits, x_up_bits))


def quantize_weights_b128(w_bits):
    """[E, K, N] bf16 bits -> codes [E, K, N] and scale codes [E, K blocks, N blocks]."""
    w = np.asarray(bf16_decode(w_bits), np.float64)
    E, K, N = w.shape
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    s = np.zeros((E, kb, nb), np.uint8)
    for e in range(E):
        for a in range(kb):
            for b in range(nb):
                t = w[e, a * BLOCK:(a + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
                s[e, a, b] = scale_codes(_amax(t.reshape(1, -1), 1))[0]
    full = np.repeat(np.repeat(s, BLOCK, axis=1)[:, :K], BLOCK, axis=2)[:, :, :N]
    return _codes(w, full), s


def groups(group_sizes, g0, El, M):
    """First rows and row counts of the local groups, rows past M left out."""
    gs = np.maximum(np.asarray(group_sizes, np.int64)[g0:g0 + El], 0)
    off = np.minimum(np.concatenate([[0], np.cumsum(gs)]), M)
    return off[:-1], np.diff(off)


def quantize_cols_b128(v, group_sizes, g0, El, M, cols):
    """Sorted rows v [M, C] (float64): codes [C, cols], scale codes [cols / 128, C],
    and which columns are written."""
    C = v.shape[1]
    qt, st, written = np.zeros((C, cols), np.uint8), np.zeros((cols // BLOCK, C), np.uint8), np.zeros(cols, bool)
    p = 0
    for r0, m in zip(*groups(group_sizes, g0, El, M)):
        for b in range(-(-int(m) // BLOCK)):
            rows = v[r0 + b * BLOCK:r0 + min(m, (b + 1) * BLOCK)]
            s = scale_codes(_amax(rows, 0))
            st[p // BLOCK] = s
            qt[:, p:p + rows.shape[0]] = _codes(rows, s[None]).T
            written[p:p + BLOCK] = True
            p += BLOCK
    return qt, st, written


def blocks_of(qt):
    """Codes [C, cols] as the calls lay them out: [cols / 128, C, 128]."""
    C, cols = qt.shape
    return np.ascontiguousarray(qt.reshape(C, cols // BLOCK, BLOCK).transpose(1, 0, 2))


def columns_of(blocks):
    """The way back."""
    n, C, _ = blocks.shape
    return np.ascontiguousarray(blocks.transpose(1, 0, 2)).reshape(C, n * BLOCK)


def spread(s, n):
    """Block scales [..., blocks] over n elements of the last axis."""
    return np.repeat(s, BLOCK, axis=-1)[..., :n]


def gmm_b128(lhs, lhs_scale, rhs, rhs_scale, group_sizes, g0, El, M):
    """lhs [M, K] codes with scale codes [M, kb]; rhs [El, N, K] codes with
    scales [El, kb, nb] (uint8 codes or float32).  The float64 result and the
    same sums on absolute values."""
    K, N = lhs.shape[1], rhs.shape[1]
    X = e4m3_decode(lhs) * spread(scale_values(lhs_scale), K)
    out, A = np.zeros((M, N)), np.zeros((M, N))
    for g, (r, m) in enumerate(zip(*groups(group_sizes, g0, El, M))):
        if m:
            W = weight_values(rhs[g], rhs_scale[g])
            out[r:r + m] = X[r:r + m] @ W.T
            A[r:r + m] = np.abs(X[r:r + m]) @ np.abs(W.T)
    return out, A


def weight_values(q, s):
    """One weight [N, K] with scales [kb, nb]."""
    N, K = q.shape
    s = scale_values(s) if s.dtype == np.uint8 else s.astype(np.float64)
    return e4m3_decode(q) * spread(np.repeat(s, BLOCK, axis=1)[:, :N].T, K)


def tgmm_b128(lhs_t, lhs_scale, rhs_t, rhs_scale, group_sizes, g0, El, M):
    """[El, K, N] float64 and the sums on absolute values."""
    K, N = lhs_t.shape[0], rhs_t.shape[0]
    out, A = np.zeros((El, K, N)), np.zeros((El, K, N))
    p = 0
    for g, (_, m) in enumerate(zip(*groups(group_sizes, g0, El, M))):
        n = BLOCK * -(-int(m) // BLOCK)
        if n:
            x = e4m3_decode(lhs_t[:, p:p + n]) * spread(scale_values(lhs_scale[p // BLOCK:(p + n) // BLOCK]).T, n)
            y = e4m3_decode(rhs_t[:, p:p + n]) * spread(scale_values(rhs_scale[p // BLOCK:(p + n) // BLOCK]).T, n)
            out[g], A[g] = x @ y.T, np.abs(x) @ np.abs(y).T
        p += n
    return out, A
