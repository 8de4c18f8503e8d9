"""The balance loss and its gradient to float32's precision: tokens of two experts,
each a sequence of its own, the rarer one chosen, so that the loss is twice
that expert's share and no sum hides an error.

Tolerances (u = 2^-24), for logits whose differences are exact.  An exponential
is within 2 ulp, 4 u, an inverse within u.  Softmax: 4 u, the sum, its inverse, the product
and the loss u each: 8 u.  Sigmoid scores exp(z) / (1 + exp(z)) for z < 0: exp(z) 4 u, the
denominator 2 u (half of an exponential's 4 u at most) + u, its inverse u and a product u, 9 u;
the other score 4 u, then 4 u as above: 17 u.  The gradient is twice p (1 - p)
(times 1 - sigmoid): p as above less the loss's u; the difference of
the counts from their mean weighted by the shares: at most 8 u of magnitudes
below 1, where 1 - p is above 0.98; two or three more products; for sigmoids 1 - sigma 4 u:
24 u and 40 u."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from tests.parity import dev_i32, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("experts", [2, 200])               # sixteen lanes a token, and a wave
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", [m.MOE_SCORE_SOFTMAX, m.MOE_SCORE_SIGMOID])
def test_shares_of_far_logits(score, dtype, experts):
    a = np.arange(4, 86, 0.5)                               # exact in bf16, and so are the differences
    n, E, top = len(a), experts, 0.0 if score == m.MOE_SCORE_SOFTMAX else 2.0
    z = np.full((n, E), -np.inf, np.float32)                # any further experts are out of service
    z[:, 0], z[:, 1] = top, -a
    if score == m.MOE_SCORE_SOFTMAX:
        p = 1 / (1 + np.exp(a))
        rest = np.ones(n)
    else:
        s0, s1 = 1 / (1 + np.exp(-top)), 1 / (1 + np.exp(a))
        p, rest = s1 / (s0 + s1), 1 - s1
    zt = torch.from_numpy(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    dt, off = (m.MOE_BF16 if dtype == "bf16" else m.MOE_F32), dev_i32(np.arange(n + 1))
    loss, counts, tokens = torch.zeros(n, device="cuda"), torch.zeros(n, E, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    m.moe_balance_loss(zt, dt, E, dev_i32(np.ones((n, 1))), n, E, 1, score, off, n, loss, counts, tokens, m.workspace(m.MOE_OP_BALANCE, n, n, 0, E))
    assert (host(counts)[:, 1] == 1).all() and (host(tokens) == 1).all()
    err = np.abs(host(loss).astype(np.float64) / (E * p) - 1)
    print("loss: at most %.1f u, at %.1f" % (err.max() / U, a[err.argmax()]), flush=True)
    assert (err <= (8 if score == m.MOE_SCORE_SOFTMAX else 17) * U).all()
    dz = torch.zeros_like(zt)
    m.moe_balance_loss_backward(zt, dt, E, counts, tokens, torch.ones(n, device="cuda"), n, E, 1, score, off, n, 0, dz, E)
    want = E * p * (1 - p) * rest
    err = np.abs(dz[:, 1].float().cpu().numpy().astype(np.float64) / want - 1)
    lim = (24 if score == m.MOE_SCORE_SOFTMAX else 40) * U
    print("gradient: at most %.1f u, at %.1f" % (err.max() / U, a[err.argmax()]), flush=True)
    assert (err <= (lim if dtype == "f32" else 2.0 ** -8 + 2 * lim)).all()
