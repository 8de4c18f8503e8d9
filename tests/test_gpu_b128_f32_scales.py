"""The grouped product in blocks of 128 with float32 weight scales at the ends of
their range, the same in every kernel: zeros, subnormals, the largest value,
infinities and NaN, in the first, a middle and the last block of a
contraction and in all of them, with ordinary blocks behind them; and
activations' scales whose product with a block leaves float32's range where the
weights' scale brings it back.

The definition: scale times block sum, added up; an infinite scale is NaN, and a
scale of zero over a NaN gives NaN.  The elements of a row or column have
one sign.  Tolerances as derived in test_gpu_b128_kernels.py."""

import pytest
import torch

import moe_fp8_grouped_amd as m
from tests.test_gpu_b128_kernels import F32_MAX, ONE_GROUP, check_product, gen, ident, operands, product

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

SPECIAL = [  # scale, by how many powers of two the rows' scales are moved, the scale of every other block of column block 3
    (0.0, 0, None), (-0.0, 0, None), (2.0 ** -149, 60, None), (1.75 * 2.0 ** -127, 60, None), (-(2.0 ** -130), 60, None),
    (2.0 ** -126, 60, None), (2.0 ** -149, 0, 2.0 ** 100), (-3 * 2.0 ** -149, 0, 2.0 ** 100), (F32_MAX, -40, None), (-F32_MAX, -40, 1.0),
    (INF, 0, None), (-INF, 0, 2.0 ** -140), (NAN, 0, None), (0.0, 60, 2.0 ** -149),
]


def positive(case, g):
    """Operands whose sums have one sign: rows positive, columns of either sign."""
    x, xs, w, ws = operands(case, m.MOE_F32, g)
    x &= 0x7F
    w &= 0x7F
    w[:, ::3] |= 0x80
    return x, xs, w, ws


@pytest.mark.parametrize("special", SPECIAL, ids=str)
@pytest.mark.parametrize("case", ONE_GROUP, ids=ident)
def test_scales_at_the_ends_of_their_range(case, special):
    print(ident(case), special, flush=True)
    s, move, other = special
    x, xs, w, ws = positive(case, gen(7))
    xs += 256 + move if move < 0 else move                  # (bytes wrap)
    x[0, 128 * 9 + 3] = 0x7F                                # NaN meets the special block too, in a row
    w[0, 140, 128 * 9 + 70] = w[0, 385, 3] = 0xFF           # and in columns
    last = ws.shape[1] - 1
    ws[0, 0, 0] = ws[0, 9, 1] = ws[0, last, 2] = s
    ws[0, :, 3] = s
    if other is not None:
        ws[0, ::2, 3] = other
    got = product(case, m.MOE_F32, m.MOE_F32, x, xs, w, ws)
    check_product(case, m.MOE_F32, x, xs, w, torch.where(ws.isinf(), NAN, ws), got)
    if s in (INF, -INF) or s != s:
        assert got[:, :384].isnan().all()


@pytest.mark.parametrize("code,factor", [(242, 2.0 ** -60), (254, 2.0 ** -100), (1, 2.0 ** 90)])
@pytest.mark.parametrize("case", ONE_GROUP, ids=ident)
def test_far_scales_of_the_rows(case, code, factor):
    print(ident(case), code, flush=True)
    x, xs, w, ws = positive(case, gen(8))
    xs.fill_(code)
    ws = (1 + torch.rand(ws.shape, generator=gen(9), device="cuda")) * factor
    check_product(case, m.MOE_F32, x, xs, w, ws, product(case, m.MOE_F32, m.MOE_F32, x, xs, w, ws))
