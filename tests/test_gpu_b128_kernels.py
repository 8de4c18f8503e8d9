"""The grouped product in blocks of 128 and its weight gradient, kernel by
kernel: every case names the kernel that its sizes choose (a host test asks the
rule), contractions of more than two windows of scales, scales that differ from
row to row, block to block and column to column, NaN, and more tiles than a
workgroup decodes at a time.

The oracle: the definition in float64, block by block, on the device.

Tolerances (u = 2^-24).  A float32 accumulator: an addition for every chunk of 8
products of the matrix core, each within 2 u (it may truncate) of the
magnitudes' sum A: K / 8 * 2 u.  With float32 scales, a block: few rows and
narrow tiles multiply the block's sum (u) and add it (u); wide tiles round a
quotient of two factors (u) and multiply every sum by it (u): 2 u a block in
either, K / 128 * 2 u.  Sums of eight waves, and the last change of units:
32 u.  What the core drops of a chunk's products: 7 of them lose less than 2^-13 of
2^(the chunk's largest exponent sum) each (tests/parity.py, which measured it),
so for a whole contraction at most 7 * 2^-13 sum_k 2^(e_a + e_b).  Half a step,
2^-8, where the result is bf16."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from tests.parity import dev_i32, host

pytestmark = pytest.mark.gpu
U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8
F8 = torch.float8_e4m3fn
F32_MAX = float(np.finfo(np.float32).max)

rng = np.random.default_rng(0)
PRODUCT = [  # kernel, group sizes, g0, El, K, N, spare rows
    ("few16", [3, 0, 1, 17, 2], 1, 4, 4240, 400, 2),
    ("few16", [16], 0, 1, 2192, 784, 0),
    ("few32", [29], 0, 1, 4240, 400, 0),
    ("few64", [150], 0, 1, 2192, 400, 1),
    ("narrow", [2600], 0, 1, 2192, 2064, 3),
    ("narrow", [40, 0, 65, 1] * 6, 2, 20, 4240, 1040, 5),
    ("wide", [330, 0, 700, 1, 260, 0], 0, 6, 4240, 7440, 5),
    ("wide", [7, 2600], 1, 1, 2192, 8208, 1),
    ("wide", [20] * 40, 4, 35, 2064, 2064, 0),
    # more tiles than a workgroup decodes at a time (64)
    ("wide", [int(v) for v in rng.integers(0, 4, 1000)], 0, 1000, 144, 6160, 7),
]
GRADIENT = [  # kernel, group sizes, g0, El, K, N
    ("narrow", [130, 0, 2200, 1], 0, 4, 272, 144),
    ("wide", [0, 2600, 1, 300, 128] * 4, 1, 17, 1024, 912),
]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(F8).view(torch.uint8)


def e8m0(g, low, high, *shape):
    return torch.randint(low, high, shape, generator=g, dtype=torch.uint8, device="cuda")


def scale(s):
    """float64 of e8m0 codes or float32 scales."""
    return torch.where(s == 255, torch.nan, torch.exp2(s.double() - 127)) if s.dtype == torch.uint8 else s.double()


def exponents(c):
    """2^e of codes, e that of the core's alignment (-6 for subnormals); 0 for zeros and NaN (which lose nothing)."""
    e = ((c >> 3) & 15).double()
    return torch.where((c & 127) == 0, 0.0, torch.exp2(torch.where(e == 0, -6.0, e - 7)))


def block_sums(x, xs, w, ws):
    """One group's product [m, n] of rows x [m, K], w [n, K] with scales xs [m, kb], ws [kb, nb]; its magnitudes' sum; 2^(exponents)."""
    out = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    A, E2 = torch.zeros_like(out), torch.zeros_like(out)
    xv, wv, xe, we = x.view(F8).double(), w.view(F8).double(), exponents(x), exponents(w)
    xs, ws = scale(xs), scale(ws)
    for b in range(xs.shape[1]):
        k = slice(128 * b, 128 * b + 128)
        s = xs[:, b, None]
        c = ws[b].repeat_interleave(128)[:w.shape[0]]
        out += c * (s * (xv[:, k] @ wv[:, k].t()))
        A += c.abs() * (s * (xv[:, k].abs() @ wv[:, k].abs().t()))
        E2 += c.abs() * (s * (xe[:, k] @ we[:, k].t()))
    return out, A, E2


def check(got, out, A, E2, K, bf16, what):
    """NaN and infinities where the definition has them (or leaves float32's range), and the rest within the tolerance."""
    got = got.double()
    lim = (K / 4 + K / 64 + 32) * U * A + 7 * 2.0 ** -13 * E2
    lim = lim + (HALF_BF16 if bf16 else U) * (out.abs() + lim) + 1e-38
    want = torch.where(out.abs() > F32_MAX, torch.copysign(torch.full_like(out, float("inf")), out), out)
    fin = torch.isfinite(want)
    bad = torch.where(fin, ~((got - want).abs() <= lim), ~((got == want) | (got.isnan() & want.isnan())))
    assert not bad.any(), (what, int(bad.sum()), [(i, float(got[tuple(i)]), float(want[tuple(i)]), float(lim[tuple(i)])) for i in bad.nonzero()[:4].tolist()])


def product(case, sdt, dtype, x, xs, w, ws, first_byte=0):
    """The call's result [M, N]; first_byte: where the weights' e8m0 scales begin in a word."""
    _, gs, g0, El, K, N, spare = case
    M, kb = x.shape[0], -(-K // 128)
    ld, lds = K + 32, -(-kb // 16) * 16 + 16
    rows = torch.full((M, ld), 0x7F, dtype=torch.uint8, device="cuda")              # NaN codes beside the rows
    rows[:, 16:16 + K] = x
    scales = torch.full((M, lds), 0xFF, dtype=torch.uint8, device="cuda")           # and NaN scales
    scales[:, :kb] = xs
    if first_byte:
        room = torch.full((ws.numel() + 8,), 0xFF, dtype=torch.uint8, device="cuda")
        room[first_byte:first_byte + ws.numel()] = ws.flatten()
        ws = room[first_byte:first_byte + ws.numel()]
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if dtype == m.MOE_BF16 else torch.float32, device="cuda")
    work = m.workspace(m.MOE_OP_GMM_B128, M, K, N, len(gs))
    m.moe_gmm_b128(rows[:, 16:16 + K], ld, scales[:, :kb], lds, w, ws, sdt, dev_i32(gs), len(gs), g0, El, M, K, N, dtype, out, work)
    assert m.moe_debug_check(work) == 0
    return out


def check_product(case, dtype, x, xs, w, ws, got):
    _, gs, g0, El, K, N, spare = case
    r = 0
    for g in range(El):
        n = gs[g0 + g]
        if n:
            check(got[r:r + n], *block_sums(x[r:r + n], xs[r:r + n], w[g], ws[g]), K, dtype == m.MOE_BF16, ("group", g))
        r += n
    assert (got[r:] == 0).all()


def operands(case, sdt, g):
    _, gs, g0, El, K, N, spare = case
    M, kb, nb = sum(gs[g0:g0 + El]) + spare, -(-K // 128), -(-N // 128)
    ws = e8m0(g, 115, 124, El, kb, nb) if sdt == m.MOE_E8M0 else (torch.rand(El, kb, nb, generator=g, device="cuda") - 0.3) * 0.01
    return codes(g, M, K), e8m0(g, 112, 126, M, kb), codes(g, El, N, K), ws


def ident(c):
    return str((c[0], len(c[1]), sum(c[1])) + tuple(c[2:]))


@pytest.mark.parametrize("dtype", [m.MOE_F32, m.MOE_BF16])
@pytest.mark.parametrize("sdt", [m.MOE_E8M0, m.MOE_F32])
@pytest.mark.parametrize("case", PRODUCT, ids=ident)
def test_product(case, sdt, dtype):
    print(ident(case), sdt, dtype, flush=True)
    x, xs, w, ws = operands(case, sdt, gen(case[4] + case[5]))
    got = product(case, sdt, dtype, x, xs, w, ws, first_byte=(case[4] // 16) % 4 if sdt == m.MOE_E8M0 else 0)
    check_product(case, dtype, x, xs, w, ws, got)


ONE_GROUP = [("few16", [9], 0, 1, 2192, 784, 0), ("few64", [64], 0, 1, 2192, 400, 0), ("narrow", [2600], 0, 1, 2192, 2064, 0),
             ("wide", [2600], 0, 1, 2192, 8208, 0)]


@pytest.mark.parametrize("sdt", [m.MOE_E8M0, m.MOE_F32])
@pytest.mark.parametrize("case", ONE_GROUP, ids=ident)
def test_nan_blocks_reach_their_results_and_no_others(case, sdt):
    """Blocks 0, 7 and the last, past the first window of scales."""
    print(ident(case), sdt, flush=True)
    _, (M,), _, _, K, N, _ = case
    x, xs, w, ws = operands(case, sdt, gen(K))
    last = K // 128                                        # (the block of 16)
    x[1, 128 * last:] = 0
    xs[1, last] = 255                                      # a NaN scale over zero codes
    xs[M - 1, 0] = 255
    x[0, 5] = 0x7F                                         # a NaN code
    w[0, 7, K - 1] = 0xFF
    ws[0, 7, 1] = 255 if sdt == m.MOE_E8M0 else float("nan")
    ws[0, last, 2] = 255 if sdt == m.MOE_E8M0 else float("nan")
    got = product(case, sdt, m.MOE_F32, x, xs, w, ws)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[[0, 1, M - 1]] = True
    want[:, 7] = True
    want[:, 128:384] = True
    assert torch.equal(got.isnan(), want)
    check_product(case, m.MOE_F32, x, xs, w, ws, got)


@pytest.mark.parametrize("case", GRADIENT, ids=ident)
def test_weight_gradient_and_its_nan_blocks(case):
    print(ident(case), flush=True)
    _, gs, g0, El, K, N = case
    M, E, g = sum(gs[g0:g0 + El]) + 3, len(gs), gen(K)
    n = m.tgmm_xt_cols(M, E) // 128
    t = [codes(g, n, C, 128) for C in (K, N)]
    s = [e8m0(g, 112, 126, n, C) for C in (K, N)]
    blocks, b = [], 0                                      # each group's first block and blocks
    for i in range(El):
        blocks.append((b, -(-gs[g0 + i] // 128)))
        b += blocks[-1][1]
    for a in t + s:                                        # what lies behind the last group is not looked at
        a[b:] = 0x7F if a.dim() == 3 else 255
    big = max(range(El), key=lambda i: gs[g0 + i])
    at = blocks[big][0] + blocks[big][1] - 1               # its last block, past the first window of scales
    t[0][at, 3, 0] = 0x7F
    s[0][blocks[big][0], K - 1] = 255
    s[1][at, 2] = 255
    dw = torch.full((El, K, N), 7.0, device="cuda")
    work = m.workspace(m.MOE_OP_TGMM_B128, M, K, N, E)
    m.moe_tgmm_b128(t[0], s[0], t[1], s[1], dev_i32(gs), E, g0, El, M, K, N, m.MOE_F32, dw, work)
    for i, (b0, nb) in enumerate(blocks):
        out, A, E2 = (torch.zeros(K, N, dtype=torch.float64, device="cuda") for _ in range(3))
        for j in range(b0, b0 + nb):
            for acc, v in ((out, lambda a: a.view(F8).double()), (A, lambda a: a.view(F8).double().abs()), (E2, exponents)):
                acc += scale(s[0][j])[:, None] * (v(t[0][j]) @ v(t[1][j]).t()) * scale(s[1][j])
        check(dw[i], out, A, E2, max(128 * nb, 1), False, ("group", i))
        want = torch.zeros(K, N, dtype=torch.bool, device="cuda")
        if i == big:
            want[[3, K - 1]] = True
            want[:, 2] = True
        assert torch.equal(dw[i].isnan(), want), i
    assert m.moe_debug_check(work) == 0


def test_narrow_tiles_of_rows_far_apart():
    """Rows of codes and scales 2^22 bytes apart, past 2^32 bytes: the same bits as of rows side by side."""
    case = NARROW_FAR
    _, (R,), _, _, K, N, _ = case
    x, xs, w, ws = operands(case, m.MOE_E8M0, gen(1))
    ld, kb, out = 1 << 22, -(-K // 128), []
    far = torch.empty(R * ld, dtype=torch.uint8, device="cuda").view(R, ld)
    near = torch.empty(R, K + 16, dtype=torch.uint8, device="cuda")
    for rows in (far, near):
        rows[:, :K], rows[:, K:K + kb] = x, xs
        l = rows.shape[1]
        out.append(torch.full((R, N), float("nan"), device="cuda"))
        m.moe_gmm_b128(rows[:, :K], l, rows[:, K:K + kb], l, w, ws, m.MOE_E8M0, dev_i32([R]), 1, 0, 1, R, K, N, m.MOE_F32, out[-1],
                       m.workspace(m.MOE_OP_GMM_B128, R, K, N, 1))
    assert torch.equal(*out)
    check_product(case, m.MOE_F32, x, xs, w, ws, out[0])


NARROW_FAR = ("narrow", [1100], 0, 1, 272, 400, 0)
