"""BlockScaledFFN with room for fewer local rows than are routed: the rows that
fit are worked on as without a limit, a slot without a row adds nothing to its
token's result and gradient and has no gradient of its own, and nothing of an
earlier step with other tokens is left.  Stage by stage against the oracle,
tolerances as in test_gpu_block_scaled_ffn.py."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from oracle import b128
from oracle import router as R
from oracle.codec import bf16_decode
from oracle.gather_reduce import gather_reduce, gather_reduce_backward
from oracle.quantize import silu_mul_backward
from tests.parity import REL_TOL, assert_bits_equal, dev_bf16, host
from tests.test_gpu_b128 import read
from tests.test_gpu_block_scaled_ffn import HALF_BF16, U, check_gmm, check_tgmm, layer, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("share", [0.0, 0.3, 0.9])
def test_rows_that_do_not_fit(share):
    T, k, E, g0, El, H, I = 150, 2, 8, 1, 6, 256, 144
    z, x, w, dout = problem(41, T, E, El, H, I)
    ids, _ = R.router_topk(bf16_decode(z), k, R.SOFTMAX, None, True, 1.0)
    gs = np.bincount(ids.reshape(-1), minlength=E)
    start, local = int(gs[:g0].sum()), int(gs[g0:g0 + El].sum())
    M = int(share * local)
    L = layer(z, x, w, k, group_offset=g0, m_cap=M)
    z2, x2, _, d2 = problem(42, T, E, 1, H, 16)              # another step first
    for a, b in ((z2, x2), (z, x)):
        L.logits.copy_(dev_bf16(a))
        L.x.copy_(dev_bf16(b))
        L.step()
        L.backward(dev_bf16(d2 if a is z2 else dout))
    torch.cuda.synchronize()
    assert np.array_equal(host(L.ids), ids) and np.array_equal(host(L.group_sizes), gs)
    rank = np.empty(T * k, np.int64)
    rank[np.argsort(ids.reshape(-1), kind="stable")] = np.arange(T * k)
    inv = (rank - start).reshape(T, k)
    inv[(inv < 0) | (inv >= M)] = -1                        # slots without a row
    got = host(L.inv_pos).reshape(T, k)
    assert np.array_equal(np.where(got < M, got, -1), inv)
    order = np.argsort(ids.reshape(-1), kind="stable")[start:start + M]
    q, s = b128.quantize_rows_b128(x)
    xq, xs = host(L.xs.q), host(L.xs.scale)
    assert np.array_equal(xq, q[order // k]) and np.array_equal(xs, s[order // k])
    assert tuple(L.ab.shape) == (M, 2 * I)
    wq = lambda w, t: (host(w.qt if t else w.q), host(w.scale_t if t else w.scale)[:, :, 0])
    y = host(L.y)
    assert not y[M:].any() and not host(L.dxs)[M:].any()
    if M:
        check_gmm(L.ab, xq, xs, *wq(L.w01, False), gs, g0, El)
        ab = host(L.ab)
        hq, hs = b128.quantize_rows_b128(ab[:, :I], ab[:, I:])
        check_gmm(L.y[:M], hq, hs, *wq(L.wo, False), gs, g0, El)
    rows = np.concatenate([y[:M], np.zeros((1, H), np.uint16)])
    g = gather_reduce(rows, True, inv, host(L.topk_w))
    lim = k * U * g["abs_sum"]
    assert (np.abs(read(L.out) - g["out"]) <= lim + HALF_BF16 * (np.abs(g["out"]) + lim) + 1e-36).all()
    b = gather_reduce_backward(dout, rows, inv, host(L.topk_w), M, M)
    dy = host(L.dy)
    assert_bits_equal(dy, b["dy"], "dy")
    dw = host(L.dw)
    assert (np.abs(dw - b["dw64"]) <= REL_TOL * b["dw_abs"]).all() and not dw[inv < 0].any()
    o, mag = R.router_topk_backward(bf16_decode(z), ids, dw, R.SOFTMAX, True, 1.0)
    lim = 288 * U * mag
    assert (np.abs(read(L.dlogits) - o) <= lim + HALF_BF16 * (np.abs(o) + lim) + 1e-36).all()
    if M == 0:
        assert not L.out.any() and not L.dx.any() and not L.dwo.any() and not L.dw01.any()
        return
    q, s = b128.quantize_rows_b128(dy)
    check_gmm(L.dh, q, s, *wq(L.wo, True), gs, g0, El)
    cols = m.tgmm_xt_cols(M, E)
    cut = lambda v: b128.quantize_cols_b128(v, gs, g0, El, M, cols)[:2]
    check_tgmm(L.dwo, *cut(b128.values(ab[:, :I], ab[:, I:])), *cut(b128.values(dy)), gs, g0, El, M, m.MOE_F32)
    da, db = silu_mul_backward(ab[:, :I], ab[:, I:], host(L.dh))
    dab = host(L.dab)
    assert_bits_equal(dab[:, :I], da, "da"), assert_bits_equal(dab[:, I:], db, "db")
    q, s = b128.quantize_rows_b128(dab)
    check_gmm(L.dxs[:M], q, s, *wq(L.w01, True), gs, g0, El)
    g = gather_reduce(np.concatenate([host(L.dxs)[:M], np.zeros((1, H), np.uint16)]), True, inv, np.ones((T, k), np.float32))
    lim = k * U * g["abs_sum"]
    assert (np.abs(read(L.dx) - g["out"]) <= lim + HALF_BF16 * (np.abs(g["out"]) + lim) + 1e-36).all()
    check_tgmm(L.dw01, *cut(b128.values(x[order // k])), *cut(b128.values(dab)), gs, g0, El, M, m.MOE_F32)
    assert m.moe_debug_check(L.ws_sort) == m.MOE_DEVERR_ROWS
