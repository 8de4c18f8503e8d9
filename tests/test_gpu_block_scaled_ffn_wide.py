"""BlockScaledFFN of a size whose products, forward and backward, run the wide
kernels: each against its definition in float64, on the codes and scales that
the device's earlier stages produced.  Tolerances as in test_gpu_b128_kernels.py."""

import pytest
import torch

import moe_fp8_grouped_amd as m
from moe_fp8_grouped_amd.pipeline import BlockScaledFFN
from tests.test_gpu_b128_kernels import F8, block_sums, check, exponents, scale

pytestmark = pytest.mark.gpu

CASE = dict(T=1500, k=2, E=10, g0=1, El=8, H=4112, I=2064)


def check_rows(L, rows, w, transposed, out, offsets):
    q, s = (w.qt, w.scale_t) if transposed else (w.q, w.scale)
    for g in range(L.El):
        a, b = offsets[g], offsets[g + 1]
        if a < b:
            check(out[a:b], *block_sums(rows.q[a:b], rows.scale[a:b], q[g], s[g, :, 0]), q.shape[2], True, ("group", g))
    assert not out[offsets[-1]:L.m_cap].any()


def check_gradient(L, x, y, dw, offsets):
    b0 = 0
    for g in range(L.El):
        nb = -(-(offsets[g + 1] - offsets[g]) // 128)
        sums = [torch.zeros(x.C, y.C, dtype=torch.float64, device="cuda") for _ in range(3)]
        for j in range(b0, b0 + nb):
            for acc, v in zip(sums, (lambda a: a.view(F8).double(), lambda a: a.view(F8).double().abs(), exponents)):
                acc += scale(x.scale[j])[:, None] * (v(x.q[j]) @ v(y.q[j]).t()) * scale(y.scale[j])
        check(dw[g], *sums, max(128 * nb, 1), dw.dtype == torch.bfloat16, ("group", g))
        b0 += nb


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
def test_every_product(grad_dtype):
    T, k, E, g0, El, H, I = (CASE[n] for n in ("T", "k", "E", "g0", "El", "H", "I"))
    g = torch.Generator(device="cuda").manual_seed(1)
    bf = lambda *s, by=1.0: (torch.randn(*s, generator=g, device="cuda") * by).to(torch.bfloat16)
    logits = bf(T, E, by=2.0)
    logits[:, 3] = -20                                      # nobody's expert among the local ones
    L = BlockScaledFFN(bf(T, H), logits, bf(El, H, I, by=0.02), bf(El, H, I, by=0.02), bf(El, I, H, by=0.02), k,
                       group_offset=g0, grad_dtype=grad_dtype, balance_weight=0.01)
    L.step()
    L.backward(bf(T, H, by=1e-3))
    sizes = L.group_sizes[g0:g0 + El].tolist()
    assert 0 in sizes and sum(sizes) < L.m_cap
    offsets = [0]
    for n in sizes:
        offsets.append(offsets[-1] + n)
    check_rows(L, L.xs, L.w01, False, L.ab, offsets)
    check_rows(L, L.hq, L.wo, False, L.y, offsets)
    check_rows(L, L.dyq, L.wo, True, L.dh, offsets)
    check_rows(L, L.dabq, L.w01, True, L.dxs, offsets)
    check_gradient(L, L.ht, L.dyt, L.dwo, offsets)
    check_gradient(L, L.xt, L.dabt, L.dw01, offsets)
    for t in (L.out, L.dx, L.dlogits):
        assert torch.isfinite(t).all() and t.any()
    for ws in (L.ws_sort, L.ws_up, L.ws_down, L.ws_balance, L.ws_dh, L.ws_dx, L.ws_dwo, L.ws_dw01):
        assert m.moe_debug_check(ws) == 0
