"""Microscaled 4-bit blocks (MXFP4 of the OCP Microscaling Formats
specification): 32 e2m1 elements, one e8m0 scale.

TEST INFRASTRUCTURE ONLY (see the package docstring).

"Keep qwix out of tpu-inference's fused MoE kernel and pre-quantize weights"
("Changes in this PR") pre-quantizes the expert weights; these are the same
weights one format further down, with a scale for every 32 elements along the
contraction instead of the page's [E, blocks, 1, N] scales.
"""

import numpy as np

from .codec import bf16_decode, e4m3_decode
from .quantize import silu_mul_f32

BLOCK = 32
# value of every code, from the format's definition
E2M1 = np.array([(-1.0 if c & 8 else 1.0) * ((c & 1) * 0.5 if (c >> 1) & 3 == 0 else
                                             (1.0 + (c & 1) * 0.5) * 2.0 ** (((c >> 1) & 3) - 1)) for c in range(16)])


def e2m1_rne(v):
    """Nearest e2m1 code of float64 values, ties to the even code, saturating."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    d = np.abs(a[..., None] - E2M1[:8])
    best = d.min(axis=-1, keepdims=True)
    tie = d == best
    even = np.arange(8) % 2 == 0
    pick = np.where((tie & even).any(-1), np.argmax(tie & even, -1), np.argmax(tie, -1))
    return (pick | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def scale_codes(blocks):
    """e8m0 codes of blocks [..., 32] (float64 values)."""
    amax = np.abs(blocks).max(axis=-1)
    with np.errstate(invalid="ignore"):
        e = np.frexp(np.where(np.isfinite(amax), amax, 1.0))[1] - 1          # floor(log2 amax)
    code = np.maximum(e - 2 + 127, 0)
    code = np.where(amax == 0, 127, code)
    return np.where(np.isfinite(blocks).all(axis=-1), code, 255).astype(np.uint8)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q):
    q = np.asarray(q, np.uint8)
    return np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[:-1] + (2 * q.shape[-1],))


def decode(q, scale):
    """float64 values of packed codes [..., C/2] and scale codes [..., C/32]."""
    s = np.where(np.asarray(scale) == 255, np.nan, np.ldexp(1.0, np.asarray(scale, np.int64) - 127))
    return E2M1[unpack(q)] * np.repeat(s, BLOCK, axis=-1)


def quantize_values(v):
    """Packed codes and scale codes of float64 rows [..., C]."""
    b = np.asarray(v, np.float64).reshape(v.shape[:-1] + (-1, BLOCK))
    s = scale_codes(b)
    y = np.where((s == 255)[..., None], 0.0, b) / np.ldexp(1.0, np.where(s == 255, 127, s).astype(np.int64) - 127)[..., None]
    return pack(e2m1_rne(y).reshape(v.shape)), s


def quantize_rows_mx4(x_bits, x_up_bits=None):
    """bf16 rows (bits) [R, C]; with x_up the float32 silu(x) * x_up."""
    x = bf16_decode(x_bits)
    return quantize_values(x if x_up_bits is None else silu_mul_f32(x, bf16_decode(x_up_bits)))


def quantize_weights_mx4(w_bits):
    """[E, K, N] -> [E, N, K/2], [E, N, K/32]."""
    return quantize_values(bf16_decode(np.ascontiguousarray(np.asarray(w_bits).transpose(0, 2, 1))))


def gmm_mx4(lhs, lhs_scale, rhs, rhs_scale, group_sizes, group_offset, num_local_experts, M=None):
    """Grouped product.  lhs e4m3 bytes with float scales ([M] or [1]), or
    packed 4-bit rows with byte scales.  Returns the float64 result and the
    same sums on absolute values."""
    lhs_scale = np.asarray(lhs_scale)
    if lhs_scale.dtype == np.uint8:
        X, ls = decode(lhs, lhs_scale), None
    else:
        X, ls = e4m3_decode(lhs), lhs_scale.astype(np.float64).reshape(-1)
    M = X.shape[0] if M is None else M
    N = rhs.shape[1]
    out, A = np.zeros((M, N)), np.zeros((M, N))
    gs = np.asarray(group_sizes, np.int64)[group_offset:group_offset + num_local_experts]
    offs = np.concatenate([[0], np.cumsum(gs)])
    for g in range(num_local_experts):
        a, b = min(int(offs[g]), M), min(int(offs[g + 1]), M)
        if a == b:
            continue
        W = decode(rhs[g], rhs_scale[g]).T
        s = 1.0 if ls is None else (ls[a:b, None] if ls.size > 1 else ls[0])
        out[a:b] = s * (X[a:b] @ W)
        A[a:b] = np.abs(s) * (np.abs(X[a:b]) @ np.abs(W))
    return out, A
