"""GPU parity of the layer from the router's logits with 4-bit expert weights
(RoutedFFN), stage by stage: every stage is checked against the oracle on the
inputs that the device's earlier stages produced, so no error is carried.

Tolerances: codes, scales, ids, rows and group sizes bit-exact.  Weights and
their gradient: the router's (logits within +-16, so a span D <= 32 and
(2 D + 64) u = 128 u of a weight, (4 D + 160) u = 288 u of the gradient's
terms, u = 2^-24).  Products: 1e-5 of the sum of magnitudes (tests/parity.py
rule 2) and half a bf16 step, 2^-8; with e4m3 rows the most that the matrix
cores' chunk rule can lose as well (HW_MAX_ERR_OVER_A).  The combine: k
float32 fmas, k u of the magnitudes, and half a bf16 step.  The few-token
layer: the oracle's own."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from moe_fp8_grouped_amd.pipeline import RoutedFFN
from oracle import mx4
from oracle import router as R
from oracle.codec import bf16_decode
from oracle.ffn_tokens import ffn_tokens
from oracle.gather_reduce import gather_reduce, gather_reduce_backward
from oracle.quantize import SCALE_ROW_DYNAMIC, quantize_rows
from tests.parity import HW_MAX_ERR_OVER_A, REL_TOL, dev_bf16, host
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu
U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8


def problem(seed, T, E, El, H, I):
    rng = np.random.default_rng(seed)
    z = to_bf16_bits(np.clip(rng.standard_normal((T, E)) * 2, -8, 8).astype(np.float32))
    x = to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    w = [to_bf16_bits((rng.standard_normal(s) * 0.05).astype(np.float32)) for s in ((El, H, I), (El, H, I), (El, I, H))]
    return z, x, w


def layer(z, x, w, k, **kw):
    return RoutedFFN(dev_bf16(x), dev_bf16(z), *(dev_bf16(v) for v in w), k, **kw)


def check_routing(L, z, k, score, renorm, scale):
    ids, tw = R.router_topk(bf16_decode(z), k, score, None, renorm, scale)
    assert np.array_equal(host(L.ids), ids)
    assert (np.abs(host(L.topk_w) - tw) <= 128 * U * tw + 1e-36).all()
    return ids


def check_product(got, lhs, ls, w, gs, g0, El, mx):
    o, A = mx4.gmm_mx4(lhs, ls, host(w.q), host(w.scale), gs, g0, El)
    lim = (REL_TOL if mx else REL_TOL + HW_MAX_ERR_OVER_A) * A
    err = np.abs(bf16_decode(host(got)).astype(np.float64) - o)
    assert (err <= lim + HALF_BF16 * (np.abs(o) + lim)).all()


CASES = [  # rows, T, k, E, g0, El, H, I, score, renormalize, scale
    (m.MOE_MX4, 97, 4, 16, 0, 16, 544, 288, R.SOFTMAX, True, 1.0),
    (m.MOE_E4M3FN, 97, 4, 16, 0, 16, 544, 288, R.SOFTMAX, False, 1.0),
    (m.MOE_MX4, 130, 6, 24, 8, 8, 256, 160, R.SIGMOID, True, 2.5),
    (m.MOE_E4M3FN, 65, 2, 8, 2, 5, 512, 96, R.SIGMOID, False, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_stages(case):
    rows, T, k, E, g0, El, H, I, score, renorm, scale = case
    z, x, w = problem([T, E], T, E, El, H, I)
    L = layer(z, x, w, k, rows=rows, few=False, score=score, renormalize=renorm, weight_scale=scale, group_offset=g0)
    for wd, wb in ((L.w01, np.concatenate([w[0], w[1]], axis=2)), (L.wo, w[2])):
        q, s = mx4.quantize_weights_mx4(wb)
        assert np.array_equal(host(wd.q), q) and np.array_equal(host(wd.scale), s)
    L.step()
    ids = check_routing(L, z, k, score, renorm, scale)
    # the sort, and the rows it moved
    order = np.argsort(ids.reshape(-1), kind="stable")
    gs = np.bincount(ids.reshape(-1), minlength=E)
    n, start = int(gs[g0:g0 + El].sum()), int(gs[:g0].sum())
    local = order[start:start + n]
    assert np.array_equal(host(L.perm), order) and np.array_equal(host(L.group_sizes), gs)
    mx = rows == m.MOE_MX4
    if mx:
        q, s = mx4.quantize_rows_mx4(x)
        xs, ss = host(L.xs.q), host(L.xs.scale)[:, :H // 32]
    else:
        q, s, _ = quantize_rows(x, SCALE_ROW_DYNAMIC)
        xs, ss = host(L.xs), host(L.ss)
    assert np.array_equal(xs[:n], q[local // k]) and np.array_equal(ss[:n], s[local // k])
    # the products, from the rows that are there
    check_product(L.ab, xs, ss, L.w01, gs, g0, El, mx)
    ab = host(L.ab)
    if mx:
        q, s = mx4.quantize_rows_mx4(ab[:, :I], ab[:, I:])
        hq, hs = host(L.hq.q), host(L.hq.scale)[:, :I // 32]
        assert np.array_equal(hq, q) and np.array_equal(hs, s)
    else:
        hq, hs = host(L.hq), host(L.hs)
    check_product(L.y, hq, hs, L.wo, gs, g0, El, mx)
    # the combine
    g = gather_reduce(host(L.y), True, host(L.inv_pos).reshape(T, k), host(L.topk_w))
    err = np.abs(bf16_decode(host(L.out)).astype(np.float64) - g["out"])
    lim = k * U * g["abs_sum"]
    assert (err <= lim + HALF_BF16 * (np.abs(g["out"]) + lim) + 1e-36).all()
    # the router's gradient, through the weights
    dout = to_bf16_bits(np.random.default_rng(T).standard_normal((T, H)).astype(np.float32))
    L.router_backward(dev_bf16(dout))
    b = gather_reduce_backward(dout, host(L.y), host(L.inv_pos).reshape(T, k), host(L.topk_w), L.m_cap, n)
    assert (np.abs(host(L.dw) - b["dw64"]) <= REL_TOL * b["dw_abs"]).all()
    o, mag = R.router_topk_backward(bf16_decode(z), ids, host(L.dw), score, renorm, scale)
    err = np.abs(bf16_decode(host(L.dlogits)).astype(np.float64) - o)
    assert (err <= 288 * U * mag + HALF_BF16 * (np.abs(o) + 288 * U * mag) + 1e-36).all()
    for ws in (L.ws_sort, L.ws_up, L.ws_down):
        assert m.moe_debug_check(ws) == 0


@pytest.mark.parametrize("T,k,g0,El", [(1, 8, 0, 16), (33, 2, 4, 8)])
def test_few_tokens(T, k, g0, El):
    E, H, I = 16, 288, 160
    z, x, w = problem([T, k], T, E, El, H, I)
    L = layer(z, x, w, k, group_offset=g0)
    assert L.few
    L.step()
    ids = check_routing(L, z, k, R.SOFTMAX, True, 1.0)
    v = [mx4.decode(host(q.q), host(q.scale)) for q in (L.w01, L.wo)]
    o, tol = ffn_tokens(x, ids, host(L.topk_w), v[0], v[1], g0, El, E)
    err = np.abs(bf16_decode(host(L.out)).astype(np.float64) - o)
    assert (err <= tol + HALF_BF16 * (np.abs(o) + tol) + 1e-36).all()
    assert m.moe_debug_check(L.ws) == 0
    with pytest.raises(ValueError):
        L.router_backward(dev_bf16(x))


def test_few_is_refused_beyond_its_sizes():
    z, x, w = problem(5, 65, 8, 8, 64, 32)
    assert not layer(z, x, w, 2).few
    with pytest.raises(ValueError):
        layer(z, x, w, 2, few=True)
    with pytest.raises(ValueError):
        layer(z, x, w, 2, rows=m.MOE_BF16)


@pytest.mark.parametrize("kw", [dict(few=True), dict(few=False), dict(few=False, rows=m.MOE_E4M3FN)], ids=str)
def test_graph_replays(kw):
    """New logits and tokens between the replays, eager steps and synchronisation of another layer's buffers too."""
    T, k, E, H, I = 48, 4, 16, 256, 128
    z, x, w = problem(7, T, E, E, H, I)
    G, eager = layer(z, x, w, k, **kw), layer(z, x, w, k, **kw)
    G.capture_graph()
    for r in range(4):
        z, x, _ = problem(100 + r, T, E, 1, H, 32)
        for L in (G, eager):
            L.x.copy_(dev_bf16(x))
            L.logits.copy_(dev_bf16(z))
        torch.cuda.synchronize()
        G.replay()
        torch.cuda.synchronize()
        eager.step()
        torch.cuda.synchronize()
        for name in ("ids", "topk_w", "out"):
            assert np.array_equal(host(getattr(G, name)), host(getattr(eager, name))), (r, name)


def test_on_another_stream_and_two_layers_at_once():
    T, k, E, H, I = 80, 4, 16, 256, 128
    z, x, w = problem(11, T, E, E, H, I)
    A, B, C = (layer(z, x, w, k) for _ in range(3))
    C.step()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            A.step()
        with torch.cuda.stream(s2):
            B.step()
    torch.cuda.synchronize()
    for L in (A, B):
        assert np.array_equal(host(L.out), host(C.out)) and np.array_equal(host(L.y), host(C.y))


@pytest.mark.parametrize("kw", [dict(few=True), dict(few=False), dict(few=False, rows=m.MOE_E4M3FN)], ids=str)
def test_no_tokens(kw):
    z, x, w = problem(3, 1, 8, 8, 64, 32)
    L = layer(z[:0], x[:0], w, 2, **kw)
    L.step()
    torch.cuda.synchronize()
    assert tuple(L.out.shape) == (0, 64)
    if not L.few:
        L.router_backward(dev_bf16(x[:0]))
        assert tuple(L.dlogits.shape) == (0, 8)
