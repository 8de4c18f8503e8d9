"""GPU parity of the training step in blocks of 128 (BlockScaledFFN), stage by
stage: every stage is checked against the oracle on the inputs that the
device's earlier stages produced, so no error is carried.

Tolerances: codes, scales, ids, rows, dy, da and db bit-exact.  Weights, their
gradient, the combine: as in the 4-bit layer's test.  Products: the b128
products' own.  The balance loss and its gradient: as in its own test; the
logits' gradient is the router's, rounded once (half a step), plus the balance
loss's, added in float32 and rounded once.

The gradients as a whole, against float64 products of the unrounded operands:
a code is off by at most 2^-4 of its value, with either sign, so that an
operand's rounding moves a product of many random terms by at most 2^-4 of its
norm.  At most eight rounded operands stand behind a gradient: x, the weights
and h on the way forward, dy, wo, dh's and x's own copies, [da | db] on the
way back; together 8 * 2^-4."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from moe_fp8_grouped_amd.pipeline import BlockScaledFFN
from oracle import b128
from oracle import balance as B
from oracle import router as R
from oracle.codec import bf16_decode
from oracle.gather_reduce import gather_reduce, gather_reduce_backward
from oracle.quantize import silu_mul_backward
from tests.parity import REL_TOL, assert_bits_equal, dev_bf16, dev_i32, host
from tests.test_gpu_b128 import exps, limits, read
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu
U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8
W = (2 * 32 + 64) * U


def problem(seed, T, E, El, H, I):
    rng = np.random.default_rng(seed)
    z = to_bf16_bits(np.clip(rng.standard_normal((T, E)) * 2, -8, 8).astype(np.float32))
    x = to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    w = [to_bf16_bits((rng.standard_normal(s) * 0.05).astype(np.float32)) for s in ((El, H, I), (El, H, I), (El, I, H))]
    return z, x, w, to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))


def layer(z, x, w, k, **kw):
    return BlockScaledFFN(dev_bf16(x), dev_bf16(z), *(dev_bf16(v) for v in w), k, **kw)


def scaled(c, s):
    """Exponent magnitudes of codes [.., K] with block scales [.., kb]."""
    return exps(c) * b128.spread(b128.scale_values(s), c.shape[-1])


def check_gmm(got, q, s, wq, ws, gs, g0, El):
    M, K, dtype = q.shape[0], q.shape[1], m.MOE_BF16
    o, A = b128.gmm_b128(q, s, wq, ws, gs, g0, El, M)
    E2 = np.zeros_like(o)
    for g, (r, c) in enumerate(zip(*b128.groups(gs, g0, El, M))):
        wsv = np.repeat(b128.scale_values(ws[g]), 128, axis=1)[:, :wq.shape[1]]
        E2[r:r + c] = scaled(q[r:r + c], s[r:r + c]) @ (exps(wq[g]) * b128.spread(wsv.T, K)).T
    assert (np.abs(read(got) - o) <= limits(o, A, K, E2, dtype)).all()


def check_tgmm(got, xq, xs, yq, ys, gs, g0, El, M, dtype):
    o, A = b128.tgmm_b128(xq, xs, yq, ys, gs, g0, El, M)
    E2, p = np.zeros_like(o), 0
    for g, (_, c) in enumerate(zip(*b128.groups(gs, g0, El, M))):
        n = 128 * -(-int(c) // 128)
        b = slice(p // 128, (p + n) // 128)
        E2[g] = scaled(xq[:, p:p + n], xs[b].T) @ scaled(yq[:, p:p + n], ys[b].T).T
        p += n
    assert (np.abs(read(got) - o) <= limits(o, A, M + 128, E2, dtype)).all()


CASES = [  # T, k, E, g0, El, H, I, score, renormalize, scale, sequences' lengths, grad dtype
    (97, 4, 16, 0, 16, 544, 288, R.SOFTMAX, True, 1.0, None, torch.float32),
    (130, 6, 24, 8, 8, 256, 160, R.SIGMOID, True, 2.5, [64, 0, 66], torch.bfloat16),
    (1, 2, 8, 0, 8, 144, 16, R.SOFTMAX, False, 1.0, [1], torch.float32),
    (300, 2, 6, 1, 4, 272, 112, R.SIGMOID, False, 1.0, [1, 250], torch.float32),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_stages(case):
    T, k, E, g0, El, H, I, score, renorm, scale, lengths, gdt = case
    z, x, w, dout = problem([T, E], T, E, El, H, I)
    off = np.array([0, T]) if lengths is None else np.concatenate([[0], np.cumsum(lengths)])
    coef = 0.125
    L = layer(z, x, w, k, score=score, renormalize=renorm, weight_scale=scale, group_offset=g0, grad_dtype=gdt, balance_weight=coef,
              seq_offsets=None if lengths is None else dev_i32(off))
    w01 = np.concatenate([w[0], w[1]], axis=2)
    for wd, wb in ((L.w01, w01), (L.wo, w[2])):
        q, s = b128.quantize_weights_b128(wb)
        assert_bits_equal(host(wd.qt), q), assert_bits_equal(host(wd.scale)[:, :, 0], s)
        assert_bits_equal(host(wd.q), np.ascontiguousarray(q.transpose(0, 2, 1)))
        assert_bits_equal(host(wd.scale_t)[:, :, 0], np.ascontiguousarray(s.transpose(0, 2, 1)))
    L.step()
    L.backward(dev_bf16(dout))
    torch.cuda.synchronize()
    # router, balance loss
    zf = bf16_decode(z)
    ids, tw = R.router_topk(zf, k, score, None, renorm, scale)
    assert np.array_equal(host(L.ids), ids) and (np.abs(host(L.topk_w) - tw) <= 128 * U * tw + 1e-36).all()
    ol, oc, on = B.balance_loss(zf, ids, score, off)
    assert np.array_equal(host(L.counts), oc) and np.array_equal(host(L.tokens), on)
    assert (np.abs(host(L.loss) - ol) <= (W + 4 * 1024 * U) * ol).all()
    # the sort, and the rows it moved, codes and scales
    order = np.argsort(ids.reshape(-1), kind="stable")
    gs = np.bincount(ids.reshape(-1), minlength=E)
    n, start = int(gs[g0:g0 + El].sum()), int(gs[:g0].sum())
    local, M = order[start:start + n], L.m_cap
    assert np.array_equal(host(L.perm), order) and np.array_equal(host(L.group_sizes), gs)
    q, s = b128.quantize_rows_b128(x)
    xq, xs = host(L.xs.q), host(L.xs.scale)
    assert np.array_equal(xq[:n], q[local // k]) and np.array_equal(xs[:n], s[local // k])
    # the forward products
    w01q, w01s, wos = host(L.w01.q), host(L.w01.scale)[:, :, 0], host(L.wo.scale)[:, :, 0]
    check_gmm(L.ab, xq, xs, w01q, w01s, gs, g0, El)
    ab = host(L.ab)
    q, s = b128.quantize_rows_b128(ab[:, :I], ab[:, I:])
    assert np.array_equal(host(L.hq.q), q) and np.array_equal(host(L.hq.scale), s)
    check_gmm(L.y, q, s, host(L.wo.q), wos, gs, g0, El)
    inv = host(L.inv_pos).reshape(T, k)
    g = gather_reduce(host(L.y), True, inv, host(L.topk_w))
    lim = k * U * g["abs_sum"]
    assert (np.abs(read(L.out) - g["out"]) <= lim + HALF_BF16 * (np.abs(g["out"]) + lim) + 1e-36).all()
    # the combine's gradients, and the logits'
    b = gather_reduce_backward(dout, host(L.y), inv, host(L.topk_w), M, n)
    dy = host(L.dy)
    assert_bits_equal(dy, b["dy"], "dy")
    assert (np.abs(host(L.dw) - b["dw64"]) <= REL_TOL * b["dw_abs"]).all()
    o, mag = R.router_topk_backward(zf, ids, host(L.dw), score, renorm, scale)
    ob, magb = B.balance_loss_backward(zf, oc, on, np.full(len(off) - 1, np.float32(coef / (len(off) - 1))), k, score, off)
    first = 288 * U * mag + HALF_BF16 * (np.abs(o) + 288 * U * mag)
    lim = first + (4 * W + 64 * U) * magb + 2 * U * (np.abs(o) + np.abs(ob) + first)
    assert (np.abs(read(L.dlogits) - o - ob) <= lim + HALF_BF16 * (np.abs(o + ob) + lim) + 1e-36).all()
    # dh, dwo
    q, s = b128.quantize_rows_b128(dy)
    assert np.array_equal(host(L.dyq.q), q) and np.array_equal(host(L.dyq.scale), s)
    check_gmm(L.dh, q, s, host(L.wo.qt), host(L.wo.scale_t)[:, :, 0], gs, g0, El)
    cols = m.tgmm_xt_cols(M, E)

    def check_cols(t, v):
        q, s, used = b128.quantize_cols_b128(v, gs, g0, El, M, cols)
        got = b128.columns_of(host(t.q)), host(t.scale)
        assert np.array_equal(got[0][:, used], q[:, used]) and np.array_equal(got[1][used[::128]], s[used[::128]])
        return got
    ht, dyt = check_cols(L.ht, b128.values(ab[:, :I], ab[:, I:])), check_cols(L.dyt, b128.values(dy))
    gdtype = m.MOE_F32 if gdt == torch.float32 else m.MOE_BF16
    check_tgmm(L.dwo, *ht, *dyt, gs, g0, El, M, gdtype)
    # da, db, dx, dw01
    da, db = silu_mul_backward(ab[:, :I], ab[:, I:], host(L.dh))
    dab = host(L.dab)
    assert_bits_equal(dab[:, :I], da, "da"), assert_bits_equal(dab[:, I:], db, "db")
    q, s = b128.quantize_rows_b128(dab)
    assert np.array_equal(host(L.dabq.q), q) and np.array_equal(host(L.dabq.scale), s)
    check_gmm(L.dxs, q, s, host(L.w01.qt), host(L.w01.scale_t)[:, :, 0], gs, g0, El)
    g = gather_reduce(host(L.dxs), True, inv, np.ones((T, k), np.float32))
    lim = k * U * g["abs_sum"]
    assert (np.abs(read(L.dx) - g["out"]) <= lim + HALF_BF16 * (np.abs(g["out"]) + lim) + 1e-36).all()
    xt, dabt = check_cols(L.xt, b128.values(x[local // k])), check_cols(L.dabt, b128.values(dab))
    check_tgmm(L.dw01, *xt, *dabt, gs, g0, El, M, gdtype)
    for ws in (L.ws_sort, L.ws_up, L.ws_down, L.ws_balance, L.ws_dh, L.ws_dx, L.ws_dwo, L.ws_dw01):
        assert m.moe_debug_check(ws) == 0


def test_gradients_of_the_unrounded_layer():
    T, k, E, H, I = 256, 2, 4, 384, 256
    z, x, w, dout = problem(21, T, E, E, H, I)
    L = layer(z, x, w, k)
    L.step()
    L.backward(dev_bf16(dout))
    ids, tw = host(L.ids), host(L.topk_w).astype(np.float64)
    X, (w0, w1, wo), D = bf16_decode(x).astype(np.float64), (bf16_decode(v).astype(np.float64) for v in w), bf16_decode(dout).astype(np.float64)
    out, dx, dw01, dwo, dtw = np.zeros((T, H)), np.zeros((T, H)), np.zeros((E, H, 2 * I)), np.zeros((E, I, H)), np.zeros((T, k))
    for j in range(k):
        for e in range(E):
            r = np.nonzero(ids[:, j] == e)[0]
            a, b = X[r] @ w0[e], X[r] @ w1[e]
            sg = 1 / (1 + np.exp(-a))
            h = a * sg * b
            y = h @ wo[e]
            out[r] += tw[r, j, None] * y
            dtw[r, j] = (y * D[r]).sum(axis=1)
            dy = tw[r, j, None] * D[r]
            dh = dy @ wo[e].T
            dab = np.concatenate([dh * b * sg * (1 + a * (1 - sg)), dh * a * sg], axis=1)
            dwo[e] += h.T @ dy
            dw01[e] += X[r].T @ dab
            dx[r] += dab @ np.concatenate([w0[e], w1[e]], axis=1).T
    dz, _ = R.router_topk_backward(bf16_decode(z), ids, dtw.astype(np.float32), R.SOFTMAX, True, 1.0)
    for name, want in (("out", out), ("dx", dx), ("dw01", dw01), ("dwo", dwo), ("dw", dtw), ("dlogits", dz)):
        got = read(getattr(L, name))
        assert np.linalg.norm(got - want) <= 8 * 2.0 ** -4 * np.linalg.norm(want), name


def test_new_weights():
    T, k, E, H, I = 40, 2, 4, 128, 64
    z, x, w, dout = problem(31, T, E, E, H, I)
    w2 = problem(32, T, E, E, H, I)[2]
    A, C = layer(z, x, w, k), layer(z, x, w2, k)
    A.requantize(*(dev_bf16(v) for v in w2))
    for L in (A, C):
        L.step()
        L.backward(dev_bf16(dout))
    for name in ("out", "dx", "dw01", "dwo", "dlogits"):
        assert np.array_equal(host(getattr(A, name)), host(getattr(C, name))), name
    with pytest.raises(ValueError, match="wo must"):
        A.requantize(*(dev_bf16(v) for v in w2[:2]), dev_bf16(w2[0]))


RESULTS = ("ids", "topk_w", "out", "loss", "counts", "tokens", "dx", "dw01", "dwo", "dlogits")


def test_graph_replays():
    """New logits, tokens and gradients between the replays, with eager work of another layer and synchronisation."""
    T, k, E, H, I = 70, 4, 16, 256, 128
    z, x, w, d = problem(7, T, E, E, H, I)
    G, eager = (layer(z, x, w, k, balance_weight=0.01) for _ in range(2))
    dout = dev_bf16(d)
    G.capture_graph(dout)
    for r in range(4):
        z, x, _, d = problem(100 + r, T, E, 1, H, 16)
        for L in (G, eager):
            L.x.copy_(dev_bf16(x))
            L.logits.copy_(dev_bf16(z))
        dout.copy_(dev_bf16(d))
        torch.cuda.synchronize()
        G.replay()
        torch.cuda.synchronize()
        eager.step()
        eager.backward(dout)
        torch.cuda.synchronize()
        for name in RESULTS:
            assert np.array_equal(host(getattr(G, name)), host(getattr(eager, name))), (r, name)


def test_on_another_stream_and_two_layers_at_once():
    T, k, E, H, I = 80, 4, 16, 256, 128
    z, x, w, d = problem(11, T, E, E, H, I)
    A, Bl, C = (layer(z, x, w, k, balance_weight=0.01) for _ in range(3))
    dout = dev_bf16(d)
    C.step()
    C.backward(dout)
    torch.cuda.synchronize()
    for _ in range(3):
        for L, s in ((A, torch.cuda.Stream()), (Bl, torch.cuda.Stream())):
            with torch.cuda.stream(s):
                L.step()
                L.backward(dout)
        torch.cuda.synchronize()
    for L in (A, Bl):
        for name in RESULTS:
            assert np.array_equal(host(getattr(L, name)), host(getattr(C, name))), name


def test_no_tokens_and_no_local_rows():
    z, x, w, d = problem(3, 5, 8, 2, 64, 32)
    L = layer(z[:0], x[:0], w, 2, balance_weight=0.1)
    L.step()
    L.backward(dev_bf16(d[:0]))
    assert tuple(L.out.shape) == (0, 64) and not L.loss.any() and not L.dw01.any() and not L.dwo.any() and tuple(L.dlogits.shape) == (0, 8)
    z[:, 6:] = to_bf16_bits(np.full((5, 2), -9, np.float32))          # nobody chooses the local experts
    L = layer(z, x, w, 2, group_offset=6)
    L.step()
    L.backward(dev_bf16(d))
    for t in (L.out, L.dx, L.dw01, L.dwo, L.dw):
        assert not t.any()
    assert m.moe_debug_check(L.ws_sort) == 0


def test_a_backward_pass_before_any_step_and_rows_that_do_not_fit():
    T, k, E, H, I = 33, 2, 4, 64, 32
    z, x, w, d = problem(5, T, E, E, H, I)
    L = layer(z, x, w, k)
    L.backward(dev_bf16(d))
    for t in (L.dx, L.dw01, L.dwo, L.dw):
        assert not t.any()
    assert m.moe_debug_check(L.ws_dwo) == 0
    L = layer(z, x, w, k, m_cap=T)                                     # half of the rows: named, and nothing past the buffers
    L.step()
    L.backward(dev_bf16(d))
    torch.cuda.synchronize()
    assert m.moe_debug_check(L.ws_sort) & m.MOE_DEVERR_ROWS and m.moe_debug_check(L.ws_up) & m.MOE_DEVERR_ROWS
    for t in (L.out, L.dx, L.dw01, L.dwo):
        assert torch.isfinite(t.float()).all()
