"""Pins of the few-token layer's oracle: against a dense torch evaluation in
float64, and the slots that take no part."""

import numpy as np
import pytest
import torch

from oracle.codec import bf16_decode
from oracle.ffn_tokens import ffn_tokens
from workloads import to_bf16_bits


@pytest.mark.parametrize("g0,El", [(0, 6), (2, 3)])
def test_against_torch(g0, El):
    T, k, E, H, I = 5, 3, 6, 24, 16
    rng = np.random.default_rng(g0)
    xb = to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    w01, wo = rng.standard_normal((El, 2 * I, H)), rng.standard_normal((El, H, I))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    tw = rng.random((T, k)).astype(np.float32)
    got, tol = ffn_tokens(xb, ids, tw, w01, wo, g0, El, E)
    x = torch.from_numpy(bf16_decode(xb).astype(np.float64))
    want = torch.zeros(T, H, dtype=torch.float64)
    for e in range(g0, g0 + El):
        ab = x @ torch.from_numpy(w01[e - g0]).T
        y = (torch.nn.functional.silu(ab[:, :I]) * ab[:, I:]) @ torch.from_numpy(wo[e - g0]).T
        want += (torch.from_numpy(tw.astype(np.float64)) * torch.from_numpy(ids == e)).sum(1, keepdim=True) * y
    assert np.allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)
    assert (tol >= 0).all() and (tol <= 1e-2 * np.abs(got).max() + 1).all()


def test_slots_without_an_expert():
    xb = to_bf16_bits(np.ones((2, 4), np.float32))
    w01, wo = np.ones((2, 4, 4)), np.ones((2, 4, 2))
    out, tol = ffn_tokens(xb, np.array([[-1, 9], [0, 0]], np.int32), np.ones((2, 2), np.float32), w01, wo, 0, 2, 2)
    assert (out[0] == 0).all() and (tol[0] == 0).all()
    one, _ = ffn_tokens(xb[1:], np.array([[0]], np.int32), np.full((1, 1), 2.0, np.float32), w01, wo, 0, 2, 2)
    assert np.allclose(out[1], one[0])
