"""The products in blocks of 128 at the largest sizes that they accept.
Operands and tolerances as in test_gpu_b128_kernels.py."""

import pytest
import torch

import moe_fp8_grouped_amd as m
from tests.parity import dev_i32
from tests.test_gpu_b128_kernels import F8, block_sums, check, codes, e8m0, exponents, gen, scale

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sdt", [m.MOE_E8M0, m.MOE_F32])
def test_float32_results_of_the_widest_rows(sdt):
    """N = 2^22 - 16, which ends inside a wave's 64 columns: 300 rows of one tile span more than 2^32 bytes."""
    M, K, N, g = 300, 16, (1 << 22) - 16, gen(1)
    x, xs, w = codes(g, M, K), e8m0(g, 112, 126, M, 16), codes(g, 1, N, K)
    nb = -(-N // 128)
    ws = e8m0(g, 115, 124, 1, 1, nb) if sdt == m.MOE_E8M0 else torch.rand(1, 1, nb, generator=g, device="cuda") - 0.3
    out, work = torch.full((M, N), float("nan"), device="cuda"), m.workspace(m.MOE_OP_GMM_B128, M, K, N, 1)
    m.moe_gmm_b128(x, K, xs, 16, w, ws, sdt, dev_i32([M]), 1, 0, 1, M, K, N, m.MOE_F32, out, work)
    for c in range(0, N, 1 << 18):
        e = min(c + (1 << 18), N)
        check(out[:, c:e], *block_sums(x, xs[:, :1], w[0, c:e], ws[0, :, c // 128:-(-e // 128)]), K, False, c)
    assert m.moe_debug_check(work) == 0


def test_float32_weight_gradient_of_the_widest_rows():
    """256 rows of a tile span more than 15/16 of 2^32 bytes."""
    M, K, N, g = 100, 272, (1 << 22) - 16, gen(2)
    n = m.tgmm_xt_cols(M, 1) // 128
    t = [codes(g, n, C, 128) for C in (K, N)]
    s = [e8m0(g, 112, 126, n, C) for C in (K, N)]
    dw, work = torch.full((1, K, N), 7.0, device="cuda"), m.workspace(m.MOE_OP_TGMM_B128, M, K, N, 1)
    m.moe_tgmm_b128(t[0], s[0], t[1], s[1], dev_i32([M]), 1, 0, 1, M, K, N, m.MOE_F32, dw, work)
    for c in range(0, N, 1 << 18):
        e = min(c + (1 << 18), N)
        sums = [scale(s[0][0])[:, None] * (v(t[0][0]) @ v(t[1][0, c:e]).t()) * scale(s[1][0, c:e])
                for v in (lambda a: a.view(F8).double(), lambda a: a.view(F8).double().abs(), exponents)]
        check(dw[0, :, c:e], *sums, 128, False, c)
    assert m.moe_debug_check(work) == 0


def test_the_most_rows():
    """2^31 - 2 rows of 16 by 16: their results past 2^36 bytes, the last tile's rows past 2^31 - 320."""
    M, K, N, g = 2 ** 31 - 2, 16, 16, gen(3)
    at = torch.tensor([0, 321, 2 ** 30 + 5, M - 337, M - 320, M - 17, M - 1], device="cuda")
    x = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    rows, w, ws = codes(g, len(at), K), codes(g, 1, N, K), e8m0(g, 115, 124, 1, 1, 1)
    rows[:, 0], w[0, :, 0] = 0x38, 0x38                     # no row of zeros
    for i, r in enumerate(at.tolist()):
        x[r] = rows[i]
    xs = torch.full((M, 16), 125, dtype=torch.uint8, device="cuda")
    out, work = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda"), m.workspace(m.MOE_OP_GMM_B128, M, K, N, 1)
    m.moe_gmm_b128(x, K, xs, 16, w, ws, m.MOE_E8M0, dev_i32([M]), 1, 0, 1, M, K, N, m.MOE_BF16, out, work)
    assert m.moe_debug_check(work) == 0
    del x, xs
    found = []
    for a in range(0, M, 1 << 26):
        found += [a + i for i in (out[a:a + (1 << 26)] != 0).any(dim=1).nonzero()[:, 0].tolist()[:100]]
    assert found == at.tolist()
    got = torch.cat([out[r:r + 1] for r in found])
    check(got, *block_sums(rows, torch.full((len(at), 1), 125, dtype=torch.uint8, device="cuda"), w[0], ws[0]), K, True, "rows")
