"""GPU parity of the b128 format (e4m3 with a power-of-two scale for every
128 elements), its grouped product and its weight gradient.

The quantizers are bit-exact: v / scale is exact and the SiLU recipe pinned.

The products (u = 2^-24): a float32 accumulator, one addition for every chunk
of 8 products of the matrix core and at most 16 more where sums are joined,
each within 2 u (it may truncate) of the magnitudes' sum A; with float32
weight scales one rounding a block and its sum, 2 u a block.  Together
(K / 8 * 2 + K / 128 * 2 + 32) u A.  To this comes what the core drops of a chunk's products:
each less than 2^-12 of 2^(the chunk's largest exponent sum) (tests/parity.py),
formed exactly for sampled results, and bounded for all by the product of the
operands' exponents: 7 * 2^-13 sum_k 2^(e_a + e_b).  Half a bf16 step, 2^-8 of
the result, where it is bf16."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from oracle import b128
from oracle.codec import bf16_decode, e4m3_decode
from tests.parity import HW_FRAC, _exp_field, _window_max, assert_bits_equal, dev_bf16, dev_f32, dev_i32, dev_u8, host
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu
U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8


def bits(rng, *shape, scale=1.0):
    return to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


# ------------------------------------------------------------ the quantizers
def gpu_rows(xb, xu=None, ldx=None, off=0, ldq=None, lds=None):
    R, C = xb.shape
    kb = -(-C // 128)
    ldx, ldq, lds = ldx or C, ldq or C, lds or kb

    def wide(b):
        t = torch.full((R, ldx), 1e30, dtype=torch.bfloat16, device="cuda")
        t[:, off:off + C] = dev_bf16(b)
        return t[:, off:off + C]
    q = torch.full((R, ldq), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((R, lds), 0xAA, dtype=torch.uint8, device="cuda")
    m.moe_quantize_rows_b128(wide(xb), None if xu is None else wide(xu), ldx, m.MOE_ACT_NONE if xu is None else m.MOE_ACT_SILU_MUL,
                             R, C, q, ldq, s, lds)
    q, s = host(q), host(s)
    assert (q[:, C:] == 0xAA).all() and (s[:, kb:] == 0xAA).all()
    return q[:, :C], s[:, :kb]


@pytest.mark.parametrize("R,C", [(1, 16), (3, 128), (37, 2080), (5, 544), (129, 7168), (1000, 112), (2, 1040)])
def test_rows_bit_exact(R, C):
    rng = np.random.default_rng(R + C)
    xb = bits(rng, R, C, scale=3.0)
    xb[0, :16] = 0x8000                                   # -0
    if R > 2:
        xb[1] = 0                                         # a row of zeros
        xb[2, : C // 2] = bits(rng, C // 2, scale=1e-38)  # subnormals
    q, s = gpu_rows(xb)
    oq, os_ = b128.quantize_rows_b128(xb)
    assert_bits_equal(s, os_, "scales")
    assert_bits_equal(q, oq, "codes")


def test_every_bfloat16_value():
    """Every bit pattern as the largest of a block and below a largest one."""
    pat = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    rng = np.random.default_rng(0)
    x = np.zeros((65536, 256), np.uint16)
    x[:, 77] = pat                                        # alone in its block
    x[:, 128] = pat
    expo = np.minimum((pat >> 7 & 0xFF).astype(np.int64) + rng.integers(0, 18, 65536), 254)
    x[:, 255] = (expo << 7).astype(np.uint16) | rng.integers(0, 128, 65536).astype(np.uint16)
    q, s = gpu_rows(x)
    oq, os_ = b128.quantize_rows_b128(x)
    assert_bits_equal(s, os_, "scales")
    assert_bits_equal(q, oq, "codes")


def test_rows_strided_gated_and_in_one_row():
    rng = np.random.default_rng(8)
    R, C = 23, 304
    xb, xu = bits(rng, R, C), bits(rng, R, C)
    q, s = gpu_rows(xb, ldx=C + 40, off=24, ldq=C + 48, lds=7)
    oq, os_ = b128.quantize_rows_b128(xb)
    assert_bits_equal(q, oq), assert_bits_equal(s, os_)
    q, s = gpu_rows(xb, xu, ldx=C + 8, off=8)
    oq, os_ = b128.quantize_rows_b128(xb, xu)
    assert_bits_equal(s, os_, "silu scales"), assert_bits_equal(q, oq, "silu codes")
    ld = 320                                              # codes and scales in one row: 304 + 3 bytes
    row = torch.zeros(R, ld, dtype=torch.uint8, device="cuda")
    m.moe_quantize_rows_b128(dev_bf16(xb), None, C, m.MOE_ACT_NONE, R, C, row[:, :C], ld, row[:, C:C + 3], ld)
    oq, os_ = b128.quantize_rows_b128(xb)
    assert_bits_equal(host(row)[:, :C], oq), assert_bits_equal(host(row)[:, C:C + 3], os_)
    assert (host(row)[:, C + 3:] == 0).all()


@pytest.mark.parametrize("E,K,N", [(1, 16, 16), (3, 144, 80), (2, 2080, 48), (2, 256, 400), (1, 1040, 128), (5, 128, 1168)])
def test_weights_bit_exact(E, K, N):
    rng = np.random.default_rng(K + N)
    wb = bits(rng, E, K, N, scale=0.02)
    wb[0, :16, 0] = 0x8000
    wb[E - 1, K // 2, N // 2] = 0x7F80                    # one block of infinity
    if K > 128:
        wb[0, 128:] = 0                                   # blocks of zeros
    kb, nb = -(-K // 128), -(-N // 128)
    oq, os_ = b128.quantize_weights_b128(wb)
    for want in ((1, 1), (1, 0), (0, 1)):
        q = torch.full((E, N, K), 0xAA, dtype=torch.uint8, device="cuda")
        s = torch.full((E, kb, 1, nb), 0xAA, dtype=torch.uint8, device="cuda")
        qt = torch.full((E, K, N), 0xAA, dtype=torch.uint8, device="cuda")
        st = torch.full((E, nb, 1, kb), 0xAA, dtype=torch.uint8, device="cuda")
        a, b = (q, s) if want[0] else (None, None), (qt, st) if want[1] else (None, None)
        m.moe_quantize_weights_b128(dev_bf16(wb), E, K, N, *a, *b)
        if want[0]:
            assert_bits_equal(host(s)[:, :, 0], os_, "scales"), assert_bits_equal(host(q), np.ascontiguousarray(oq.transpose(0, 2, 1)), "codes")
        if want[1]:
            assert_bits_equal(host(st)[:, :, 0], np.ascontiguousarray(os_.transpose(0, 2, 1)), "scales_t")
            assert_bits_equal(host(qt), oq, "codes_t")


COLS = [  # group sizes, g0, El, C, gated, gathered (top-k)
    ([3], 0, 1, 16, False, 0),
    ([128, 0, 129, 1, 255], 0, 5, 144, False, 0),
    ([4, 0, 130, 1, 128, 60, 7, 2], 1, 5, 272, False, 2),
    ([0, 0, 0], 0, 3, 32, False, 0),
    ([70, 300, 10, 5], 1, 2, 400, True, 0),
    ([5] * 100, 7, 90, 128, False, 5),
    ([2] * 1024, 3, 1000, 48, True, 4),
]


@pytest.mark.parametrize("case", COLS, ids=lambda c: str((len(c[0]),) + c[1:]))
def test_columns_bit_exact(case):
    gs, g0, El, C, gated, k = case
    gs = np.array(gs)
    rng = np.random.default_rng(C + El)
    n, start, E = int(gs[g0:g0 + El].sum()), int(gs[:g0].sum()), len(gs)
    M = n + 13                                            # more room than rows
    cols = m.tgmm_xt_cols(M, E)
    if k:
        T = int(gs.sum()) // k
        assert T * k == gs.sum()
        xb, xu = bits(rng, T, C, scale=2.0), bits(rng, T, C)
        perm = rng.permutation(T * k).astype(np.int32)
        src = perm[start:start + n] // k
    else:
        T, k, perm = M, 1, None
        xb, xu = bits(rng, M, C, scale=2.0), bits(rng, M, C)
        src = np.arange(n)
    xb[0, : C // 2] = 0
    if T > 1:
        xb[1] = bits(rng, C, scale=1e-38)
        xb[T - 1, 3] = 0x7FC0                             # a NaN spoils one column of one block
    ldx = C + 24
    wide = [torch.full((T, ldx), 1e30, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, b in zip(wide, (xb, xu)):
        t[:, 8:8 + C] = dev_bf16(b)
    qt = torch.full((cols // 128, C, 128), 0xAA, dtype=torch.uint8, device="cuda")
    st = torch.full((cols // 128, C), 0xAA, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    m.moe_quantize_cols_b128(wide[0][:, 8:8 + C], wide[1][:, 8:8 + C] if gated else None, ldx, m.MOE_ACT_SILU_MUL if gated else m.MOE_ACT_NONE,
                             T, k, None if perm is None else dev_i32(perm), dev_i32(gs), E, g0, El, M, C, qt, st, ws)
    with np.errstate(all="ignore"):
        v = b128.values(xb[src], xu[src] if gated else None)
    oq, os_, written = b128.quantize_cols_b128(v, gs, g0, El, M, cols)
    q, s = b128.columns_of(host(qt)), host(st)
    assert_bits_equal(s[written[::128]], os_[written[::128]], "scales")
    assert_bits_equal(q[:, written], oq[:, written], "codes")
    assert (q[:, ~written] == 0xAA).all() and (s[~written[::128]] == 0xAA).all()
    assert m.moe_debug_check(ws) == 0


def test_columns_of_bad_sizes_and_indexes_stay_inside():
    C, E, M, T, k = 64, 4, 100, 40, 4
    rng = np.random.default_rng(1)
    x = dev_bf16(bits(rng, T, C))
    cols = m.tgmm_xt_cols(M, E)
    for gs, bit in (([50, -3, 30, 0], m.MOE_DEVERR_GROUP_SIZE), ([50, 60, 2 ** 31 - 1, 2 ** 31 - 1], m.MOE_DEVERR_ROWS)):
        qt = torch.zeros((cols // 128, C, 128), dtype=torch.uint8, device="cuda")
        st = torch.zeros((cols // 128, C), dtype=torch.uint8, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        perm = rng.integers(-2 ** 31, 2 ** 31, T * k).astype(np.int32)
        m.moe_quantize_cols_b128(x, None, C, m.MOE_ACT_NONE, T, k, dev_i32(perm), dev_i32(gs), E, 0, E, M, C, qt, st, ws)
        assert m.moe_debug_check(ws) == bit


# ------------------------------------------------------------ the products
def codes(rng, *shape, spread=1.0):
    """Codes as a quantizer leaves them: normal values over most of the format."""
    v = rng.standard_normal(shape) * 100 * spread
    return b128.e4m3_rne(np.clip(v, -448, 448).astype(np.float32))


def limits(out, A, K, E2, dtype):
    """Bound for every result; E2: sum_k 2^(exponents) with the scales."""
    lim = (K / 4 + K / 64 + 32) * U * A + 7 * 2.0 ** -13 * E2
    return lim + ((HALF_BF16 * (np.abs(out) + lim)) if dtype == m.MOE_BF16 else U * np.abs(out)) + 1e-38


def exps(c):
    return np.where((c & 127) == 0, 0.0, np.ldexp(1.0, _exp_field(c)))


def dropped(xc, xs, wc, ws):
    """Exactly bounded loss of sampled dot products: codes [n, K] and float scales [n, K] of both operands."""
    p = np.abs(e4m3_decode(xc) * e4m3_decode(wc))
    return (np.minimum(p, HW_FRAC * _window_max(exps(xc) * exps(wc))) * xs * ws).sum(axis=-1)


def read(t):
    a = host(t)
    return bf16_decode(a).astype(np.float64) if a.dtype == np.uint16 else a.astype(np.float64)


GMM = [  # group sizes, g0, El, K, N, spare rows
    ([1], 0, 1, 16, 16, 0),
    ([1], 0, 1, 400, 144, 0),
    ([3, 0, 1, 17], 0, 4, 272, 160, 5),
    ([2, 5, 0, 40, 1, 9], 2, 3, 144, 1040, 3),
    ([33], 0, 1, 1040, 400, 0),
    ([64, 1, 0, 130], 0, 4, 2080, 272, 0),
    ([300, 5, 257], 0, 3, 384, 528, 9),
    ([1] * 70, 0, 70, 256, 128, 0),
    ([700, 0, 530], 0, 3, 640, 1040, 0),
    ([4] * 1024, 5, 1000, 128, 32, 7),
    ([0, 0], 0, 2, 128, 64, 11),
    ([1500, 300, 260, 515], 0, 4, 1152, 1536, 1),
    ([2600], 0, 1, 528, 2064, 0),
    # as many tiles of 256 by 256 as the GPU has workgroups, and more
    ([700, 300, 0, 616, 1200], 0, 5, 2080, 4112, 40),
    ([9, 300, 0, 17, 1, 256, 257, 31] * 4, 1, 30, 528, 2320, 5),
    ([513, 0, 40] * 4, 3, 7, 16, 7184, 0),
]


@pytest.mark.parametrize("dtype", [m.MOE_F32, m.MOE_BF16])
@pytest.mark.parametrize("sdt", [m.MOE_E8M0, m.MOE_F32])
@pytest.mark.parametrize("case", GMM, ids=lambda c: str((len(c[0]), sum(c[0])) + c[1:]))
def test_product(case, sdt, dtype):
    gs, g0, El, K, N, spare = case
    print(case, sdt, dtype, flush=True)
    gs = np.array(gs)
    rng = np.random.default_rng(K + N)
    n, E = int(gs[g0:g0 + El].sum()), len(gs)
    M, kb, nb = n + spare, -(-K // 128), -(-N // 128)
    x, w = codes(rng, M, K), codes(rng, El, N, K)
    xs = rng.integers(115, 124, (M, kb)).astype(np.uint8)
    ws = rng.integers(115, 124, (El, kb, nb)).astype(np.uint8) if sdt == m.MOE_E8M0 else ((rng.random((El, kb, nb)) - 0.3) * 0.01).astype(np.float32)
    ld, lds = K + 32, -(-kb // 16) * 16 + 16
    rows = torch.full((M, ld), 0x7F, dtype=torch.uint8, device="cuda")              # NaN codes beside the rows
    rows[:, 16:16 + K] = dev_u8(x)
    scales = torch.full((M, lds), 0xFF, dtype=torch.uint8, device="cuda")           # and NaN scales
    scales[:, :kb] = dev_u8(xs)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if dtype == m.MOE_BF16 else torch.float32, device="cuda")
    work = m.workspace(m.MOE_OP_GMM_B128, M, K, N, E)
    m.moe_gmm_b128(rows[:, 16:16 + K], ld, scales[:, :kb], lds, dev_u8(w), (dev_u8 if sdt == m.MOE_E8M0 else dev_f32)(ws), sdt, dev_i32(gs), E, g0, El,
                   M, K, N, dtype, out, work)
    got = read(out)
    assert (got[n:] == 0).all()
    o, A = b128.gmm_b128(x, xs, w, ws, gs, g0, El, M)
    wsv = np.abs(b128.scale_values(ws) if ws.dtype == np.uint8 else ws.astype(np.float64))
    X2 = exps(x) * b128.spread(b128.scale_values(xs), K)
    group = np.repeat(np.arange(El), gs[g0:g0 + El])
    W2 = [exps(w[g]) * b128.spread(np.repeat(wsv[g], 128, axis=1)[:, :N].T, K) for g in range(El)]
    E2 = np.zeros((M, N))
    for g, (r, c) in enumerate(zip(*b128.groups(gs, g0, El, M))):
        E2[r:r + c] = X2[r:r + c] @ W2[g].T
    err = np.abs(got - o)
    assert (err <= limits(o, A, K, E2, dtype)).all()
    # sampled results against the exact bound of what the core drops
    if n:
        r, c = rng.integers(0, n, 400), rng.integers(0, N, 400)
        r[:4], c[:4] = (0, n - 1, 0, n - 1), (0, N - 1, N - 1, 0)
        g = group[r]
        one = np.ones(K)
        d = dropped(x[r], b128.spread(b128.scale_values(xs[r]), K), w[g, c], np.stack([np.repeat(wsv[gg, :, cc // 128], 128)[:K] * one for gg, cc in zip(g, c)]))
        lim = (K / 4 + K / 64 + 32) * U * A[r, c] + d
        lim = lim + (HALF_BF16 * (np.abs(o[r, c]) + lim) if dtype == m.MOE_BF16 else U * np.abs(o[r, c]))
        assert (err[r, c] <= lim).all()
    assert m.moe_debug_check(work) == 0


@pytest.mark.parametrize("M", [2, 600])
@pytest.mark.parametrize("sdt", [m.MOE_E8M0, m.MOE_F32])
def test_nan_blocks_reach_their_results_and_no_others(M, sdt):
    K, N = 400, 400
    rng = np.random.default_rng(3)
    x, w = codes(rng, M, K), codes(rng, 1, N, K)
    xs, ws = np.full((M, 4), 120, np.uint8), np.full((1, 4, 4), 120, np.uint8)
    x[1, 384:] = 0
    xs[1, 3] = 255                                        # a NaN scale over zero codes
    x[0, 5] = 0x7F                                        # a NaN code
    w[0, 7, 399] = 0xFF
    if sdt == m.MOE_E8M0:
        ws[0, 2, 1] = 255
    else:
        ws = b128.scale_values(ws).astype(np.float32)
        ws[0, 2, 1] = np.nan
    scales = torch.full((M, 16), 0x7F, dtype=torch.uint8, device="cuda")
    scales[:, :4] = dev_u8(xs)
    out = torch.zeros((M, N), device="cuda")
    m.moe_gmm_b128(dev_u8(x), K, scales[:, :4], 16, dev_u8(w), (dev_u8 if sdt == m.MOE_E8M0 else dev_f32)(ws), sdt, dev_i32([M]), 1, 0, 1, M, K, N,
                   m.MOE_F32, out, m.workspace(m.MOE_OP_GMM_B128, M, K, N, 1))
    want = np.zeros((M, N), bool)
    want[:2] = True
    want[:, 7] = True
    want[:, 128:256] = True
    assert np.array_equal(np.isnan(host(out)), want)


def test_product_names_bad_sizes_and_stays_inside():
    M, K, N, E = 50, 256, 128, 4
    rng = np.random.default_rng(4)
    x, w = dev_u8(codes(rng, M, K)), dev_u8(codes(rng, E, N, K))
    xs, ws = torch.full((M, 16), 120, dtype=torch.uint8, device="cuda"), torch.full((E, 2, 1), 120, dtype=torch.uint8, device="cuda")
    for gs, bit in (([20, -3, 10, 0], m.MOE_DEVERR_GROUP_SIZE), ([20, 40, 2 ** 31 - 1, 2 ** 31 - 1], m.MOE_DEVERR_ROWS)):
        out, work = torch.zeros((M, N), device="cuda"), m.workspace(m.MOE_OP_GMM_B128, M, K, N, E)
        m.moe_gmm_b128(x, K, xs, 16, w, ws, m.MOE_E8M0, dev_i32(gs), E, 0, E, M, K, N, m.MOE_F32, out, work)
        assert m.moe_debug_check(work) == bit
        dw, work = torch.zeros((E, K, N), device="cuda"), m.workspace(m.MOE_OP_TGMM_B128, M, K, N, E)
        cols = m.tgmm_xt_cols(M, E)
        t = [torch.full((cols // 128, c, 128), 0x38, dtype=torch.uint8, device="cuda") for c in (K, N)]
        s = [torch.full((cols // 128, c), 120, dtype=torch.uint8, device="cuda") for c in (K, N)]
        m.moe_tgmm_b128(t[0], s[0], t[1], s[1], dev_i32(gs), E, 0, E, M, K, N, m.MOE_F32, dw, work)
        assert m.moe_debug_check(work) == bit


TGMM = [  # group sizes, g0, El, K, N
    ([1], 0, 1, 16, 16),
    ([3, 0, 130, 1], 0, 4, 144, 80),
    ([5, 200, 0, 128, 129, 64, 3], 1, 5, 272, 400),
    ([0, 0], 0, 2, 48, 32),
    ([700, 300], 0, 2, 528, 1040),
    ([40] * 20, 3, 15, 256, 128),
    ([2] * 1024, 3, 1000, 16, 32),
    ([256, 1, 513, 0, 384], 0, 5, 768, 512),
    ([2000], 0, 1, 1040, 272),
    ([0, 2100, 1, 0, 0, 128, 129, 255, 600, 0] * 2, 0, 20, 784, 1040),
    ([300] * 17, 0, 17, 1024, 1024),
]


@pytest.mark.parametrize("dtype", [m.MOE_F32, m.MOE_BF16])
@pytest.mark.parametrize("case", TGMM, ids=lambda c: str((len(c[0]), sum(c[0])) + c[1:]))
def test_weight_gradient(case, dtype):
    gs, g0, El, K, N = case
    print(case, dtype, flush=True)
    gs = np.array(gs)
    rng = np.random.default_rng(K + N)
    n, E = int(gs[g0:g0 + El].sum()), len(gs)
    M = n + 3
    cols = m.tgmm_xt_cols(M, E)
    q, s = [], []
    for C in (K, N):
        v = rng.standard_normal((M, C)) * np.exp(rng.uniform(-3, 3, C))
        a, b, written = b128.quantize_cols_b128(v, gs, g0, El, M, cols)
        a[:, ~written], b[~written[::128]] = 0x7F, 255      # what lies behind the last group is not looked at
        q.append(a), s.append(b)
    out = torch.full((El, K, N), float("nan"), dtype=torch.bfloat16 if dtype == m.MOE_BF16 else torch.float32, device="cuda")
    work = m.workspace(m.MOE_OP_TGMM_B128, M, K, N, E)
    m.moe_tgmm_b128(dev_u8(b128.blocks_of(q[0])), dev_u8(s[0]), dev_u8(b128.blocks_of(q[1])), dev_u8(s[1]), dev_i32(gs), E, g0, El, M, K, N, dtype, out, work)
    got = read(out)
    o, A = b128.tgmm_b128(q[0], s[0], q[1], s[1], gs, g0, El, M)
    p = 0
    for g, (_, c) in enumerate(zip(*b128.groups(gs, g0, El, M))):
        L = 128 * -(-int(c) // 128)
        sc = [b128.spread(b128.scale_values(b[p // 128:(p + L) // 128]).T, L) for b in s]
        E2 = (exps(q[0][:, p:p + L]) * sc[0]) @ (exps(q[1][:, p:p + L]) * sc[1]).T
        err = np.abs(got[g] - o[g])
        assert (err <= limits(o[g], A[g], max(L, 1), E2, dtype)).all(), g
        if L and g % 50 == 0:
            r, t = rng.integers(0, K, 200), rng.integers(0, N, 200)
            d = dropped(q[0][r, p:p + L], sc[0][r], q[1][t, p:p + L], sc[1][t])
            lim = (L / 4 + L / 64 + 32) * U * A[g][r, t] + d
            lim = lim + (HALF_BF16 * (np.abs(o[g][r, t]) + lim) if dtype == m.MOE_BF16 else U * np.abs(o[g][r, t])) + 1e-38
            assert (err[r, t] <= lim).all(), g
        p += L
    assert m.moe_debug_check(work) == 0


def test_a_window_without_experts_or_rows():
    rng = np.random.default_rng(5)
    x, xs = dev_u8(codes(rng, 5, 128)), torch.full((5, 16), 120, dtype=torch.uint8, device="cuda")
    out = torch.full((5, 32), 7.0, device="cuda")
    ws = m.workspace(m.MOE_OP_GMM_B128, 5, 128, 32, 4)
    m.moe_gmm_b128(x, 128, xs, 16, None, None, m.MOE_E8M0, dev_i32([1, 1, 1, 2]), 4, 4, 0, 5, 128, 32, m.MOE_F32, out, ws)
    assert (host(out) == 0).all()
    dw = torch.full((2, 32, 16), 7.0, device="cuda")
    m.moe_tgmm_b128(None, None, None, None, dev_i32([0, 0]), 2, 0, 2, 0, 32, 16, m.MOE_F32, dw, m.workspace(m.MOE_OP_TGMM_B128, 0, 32, 16, 2))
    assert (host(dw) == 0).all()


@pytest.mark.parametrize("M,El", [(3, 8), (700, 2)])
def test_the_same_bits_every_time_and_in_a_graph(M, El):
    K, N = 528, 784
    rng = np.random.default_rng(M)
    gs = dev_i32([M // El + (i < M % El) for i in range(El)])
    xb = dev_bf16(bits(rng, M, K))
    dyb = dev_bf16(bits(rng, M, N, scale=1e-3))
    w = dev_bf16(bits(rng, El, K, N, scale=0.02))
    kb, nb, cols = -(-K // 128), -(-N // 128), m.tgmm_xt_cols(M, El)
    u8 = dict(dtype=torch.uint8, device="cuda")
    b = dict(q=torch.zeros(M, K + 16, **u8), wq=torch.zeros(El, N, K, **u8), ws=torch.zeros(El, kb, 1, nb, **u8), wt=torch.zeros(El, K, N, **u8),
             wst=torch.zeros(El, nb, 1, kb, **u8), xt=torch.zeros(cols // 128, K, 128, **u8), xts=torch.zeros(cols // 128, K, **u8), yt=torch.zeros(cols // 128, N, 128, **u8),
             yts=torch.zeros(cols // 128, N, **u8), y=torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), dw=torch.zeros(El, K, N, device="cuda"))
    work, twork = m.workspace(m.MOE_OP_GMM_B128, M, K, N, El), m.workspace(m.MOE_OP_TGMM_B128, M, K, N, El)
    x = torch.empty_like(xb)

    def call():
        m.moe_quantize_rows_b128(x, None, K, 0, M, K, b["q"][:, :K], K + 16, b["q"][:, K:K + kb], K + 16)
        m.moe_quantize_weights_b128(w, El, K, N, b["wq"], b["ws"], b["wt"], b["wst"])
        m.moe_gmm_b128(b["q"][:, :K], K + 16, b["q"][:, K:K + kb], K + 16, b["wq"], b["ws"], m.MOE_E8M0, gs, El, 0, El, M, K, N, m.MOE_BF16, b["y"], work)
        m.moe_quantize_cols_b128(x, None, K, 0, M, 1, None, gs, El, 0, El, M, K, b["xt"], b["xts"], twork)
        m.moe_quantize_cols_b128(dyb, None, N, 0, M, 1, None, gs, El, 0, El, M, N, b["yt"], b["yts"], twork)
        m.moe_tgmm_b128(b["xt"], b["xts"], b["yt"], b["yts"], gs, El, 0, El, M, K, N, m.MOE_F32, b["dw"], twork)
    x.copy_(xb)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for r in range(4):
        x.copy_(xb.roll(r, 0))
        torch.cuda.synchronize()
        g.replay()
        got = {n: t.clone() for n, t in b.items()}
        torch.cuda.synchronize()
        call()
        for n, t in b.items():
            assert torch.equal(got[n], t), (r, n)
