"""Pins of the balance loss's oracle (no GPU)."""

import numpy as np
import pytest

from oracle import balance as B


def case(seed, T=40, E=6, k=2):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) * 2
    z[3] = -np.inf
    z[5, 2], z[6, 1], z[7] = -np.inf, np.nan, float(np.finfo(np.float32).min)
    ids = np.argsort(-np.where(np.isnan(z), -np.inf, z), axis=1, kind="stable")[:, :k].astype(np.int32)
    return z, ids, np.array([2, 2, 17, 18, 36])


def test_even_routing_costs_one():
    T, E, k = 24, 8, 2
    z = np.zeros((T, E))
    ids = np.stack([(np.arange(T) * k + j) % E for j in range(k)], axis=1)
    for score in (B.SOFTMAX, B.SIGMOID):
        loss, counts, tokens = B.balance_loss(z, ids, score, np.array([0, T]))
        assert np.isclose(loss[0], 1.0) and (counts[0] == T * k // E).all() and tokens[0] == T


def test_everything_to_one_expert_costs_the_number_of_experts():
    z = np.full((10, 4), -60.0)
    z[:, 3] = 60.0
    loss, counts, _ = B.balance_loss(z, np.full((10, 1), 3), B.SOFTMAX, np.array([0, 10]))
    assert np.isclose(loss[0], 4.0) and counts[0].tolist() == [0, 0, 0, 10]


def test_counts_and_tokens_leave_out_what_is_not_there():
    z, ids, off = case(0)
    ids[20, 0], ids[21] = -1, [99, 6]
    _, counts, tokens = B.balance_loss(z, ids, B.SOFTMAX, off)
    assert counts.sum(axis=1).tolist() == [0, 2 * (15 - 2), 2, 2 * 18 - 3] and tokens.tolist() == [0, 13, 1, 18]


@pytest.mark.parametrize("score", [B.SOFTMAX, B.SIGMOID])
def test_gradient_against_differences(score):
    z, ids, off = case(1)
    dl = np.array([0.5, -1.0, 2.0, 0.25])
    loss, counts, tokens = B.balance_loss(z, ids, score, off)
    dz, mag = B.balance_loss_backward(z, counts, tokens, dl, 2, score, off)
    assert (np.abs(dz) <= mag * (1 + 1e-12)).all() and (dz[:2] == 0).all() and (dz[36:] == 0).all()
    assert (dz[~B.in_service(z)] == 0).all()
    h = 1e-5
    for t, e in ((2, 0), (4, 5), (5, 1), (6, 0), (17, 3), (18, 2), (35, 4)):
        up, down = z.copy(), z.copy()
        up[t, e] += h
        down[t, e] -= h
        d = ((B.balance_loss(up, ids, score, off)[0] - B.balance_loss(down, ids, score, off)[0]) * dl).sum() / (2 * h)
        assert abs(d - dz[t, e]) <= 1e-8 + 1e-6 * mag[t, e]


def test_sigmoid_shares_far_below_zero_are_ratios():
    z = np.array([[-800.0, -800.0 + np.log(3.0)], [-200.0, -np.inf]])
    p, _ = B.shares(z, B.SIGMOID)
    assert np.allclose(p, [[0.25, 0.75], [1.0, 0.0]])
