"""Pins of the router oracle: against torch's softmax and top-k, the rules of
masked rows and ties, and the gradient against differences."""

import numpy as np
import pytest
import torch

from oracle import router as R


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_against_torch(score, renorm):
    z = torch.randn(40, 24, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    ids, w = R.router_topk(z.numpy(), 5, score, renorm=renorm, scale=2.5)
    p = torch.softmax(z, -1) if score == R.SOFTMAX else torch.sigmoid(z)
    top = torch.topk(p, 5)
    assert (top.indices.numpy() == ids).all()
    want = top.values / top.values.sum(-1, keepdim=True) if renorm else top.values
    assert np.allclose(w, 2.5 * want.numpy(), rtol=1e-13)


def test_ties_masks_and_bias():
    z = np.array([[1.0, 2.0, 2.0, 0.0], [-np.inf] * 4, [-np.inf, 3.0, np.nan, -np.inf], [0.0, 0.0, 0.0, 0.0]])
    ids, w = R.router_topk(z, 3, R.SOFTMAX)
    assert ids.tolist() == [[1, 2, 0], [0, 1, 2], [1, 0, 2], [0, 1, 2]]
    assert (w[1] == 0).all() and w[2].tolist() == [1.0, 0.0, 0.0]
    ids, w = R.router_topk(z, 2, R.SIGMOID, bias=np.array([0.9, 0.0, 0.0, 0.0]), renorm=True)
    assert ids[0].tolist() == [0, 1] and ids[1].tolist() == [0, 1] and ids[2].tolist() == [1, 0]
    assert (w[1] == 0).all() and np.isclose(w[0].sum(), 1)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    z = rng.standard_normal((4, 9))
    z[1, 3] = -np.inf
    ids, _ = R.router_topk(z, 3, score)
    ids[3] = [2, 2, 5]                                  # the same expert twice
    dw = rng.standard_normal((4, 3))
    d, mag = R.router_topk_backward(z, ids, dw, score, renorm, 1.7)
    h = 1e-6
    for t in range(4):
        for e in range(9):
            if np.isinf(z[t, e]):
                assert d[t, e] == 0
                continue
            zp, zm = z.copy(), z.copy()
            zp[t, e] += h
            zm[t, e] -= h
            f = lambda q: float((R.weights_of(q, ids, score, renorm, 1.7) * dw).sum())
            assert abs((f(zp) - f(zm)) / (2 * h) - d[t, e]) < 1e-8
    assert (mag >= np.abs(d) - 1e-12).all()
