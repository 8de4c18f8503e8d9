"""GPU parity of the router and its backward against the oracle.

Tolerances (derived, u = 2^-24): a softmax weight is exp(z - m) over a sum.
z - m is rounded once (|z - m| u on the result's logarithm), expf is within
2 ulp = 4 u, the sum of up to 1024 positive terms is a 16-term lane sum and a
6-level tree (each level u) of terms with those errors, and the quotient, the
renormalisation (the same again) and the factor add u each: a relative
(2 D + 64) u, D = the largest |z - m| of a chosen expert.  Sigmoid: expf of a
rounded argument is exact in z, so (64) u.  The gradient's terms carry two
such weights each: (4 D + 160) u of the sum of the terms' magnitudes, plus
half a bf16 step (2^-8 of the value) where the result is bf16.  Values below
2^-120 may lose bits as subnormals: 1e-36 absolute."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from oracle import router as R
from tests.parity import dev_f32, dev_i32, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NEG = float(np.finfo(np.float32).min)

CASES = [  # T, E, k, dtype, score, bias, renorm, scale
    (1, 256, 8, "f32", R.SIGMOID, True, True, 2.5),
    (1, 1, 1, "f32", R.SOFTMAX, False, True, 1.0),
    (5, 13, 3, "bf16", R.SOFTMAX, False, False, 1.0),
    (130, 64, 8, "f32", R.SOFTMAX, False, True, 1.0),
    (67, 8, 8, "bf16", R.SIGMOID, False, True, 1.5),
    (33, 1024, 64, "f32", R.SOFTMAX, True, False, 1.0),
    (257, 72, 6, "bf16", R.SIGMOID, True, False, 2.5),
    (1000, 256, 8, "bf16", R.SOFTMAX, False, False, 1.0),
    (259, 128, 4, "f32", R.SOFTMAX, True, True, 0.5),
    (17, 513, 1, "f32", R.SIGMOID, False, False, 1.0),
    (4099, 160, 6, "f32", R.SOFTMAX, False, True, 16.0),
    (3, 65, 2, "bf16", R.SOFTMAX, True, True, 1.0),
]


def draw(T, E, dtype, seed, width=None):
    """Logits with the rows that matter: masked experts, rows without any
    expert, the type's lowest value as a mask, equal logits."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, width or E)).astype(np.float32) * 2
    if T > 2:
        z[rng.random(z.shape) < 0.05] = -np.inf
        z[1::7] = -np.inf
        z[2::11] = NEG
        z[0, ::2] = NEG
        z[min(4, T - 1)] = 0.25
    t = torch.from_numpy(z)
    if dtype == "bf16":
        t = t.to(torch.bfloat16)
    return t.cuda()


def run(z, T, E, k, score, bias, renorm, scale, ldl=None):
    dt = m.MOE_BF16 if z.dtype == torch.bfloat16 else m.MOE_F32
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    m.moe_router_topk(z, dt, ldl or E, T, E, k, score, bias, int(renorm), scale, ids, w)
    return ids, w


def span(z, ids):
    """D: how far below its maximum (or the chosen maximum) a chosen finite logit lies, capped where exp is 0."""
    zc = np.take_along_axis(z, ids.astype(np.int64), -1)
    top = np.nanmax(np.where(np.isneginf(z), np.nan, z), axis=-1, initial=-np.inf, keepdims=True)
    d = np.where(np.isneginf(zc) | np.isneginf(top), 0.0, top - zc)
    return np.minimum(d, 110.0)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_topk_matches_the_oracle(case):
    T, E, k, dtype, score, has_bias, renorm, scale = case
    z = draw(T, E, dtype, 10 * E + T)
    bias = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.1 if has_bias else None
    ids, w = run(z, T, E, k, score, None if bias is None else dev_f32(bias), renorm, scale)
    zf = z.float().cpu().numpy().astype(np.float64)
    oid, ow = R.router_topk(zf, k, score, bias, renorm, scale)
    assert (host(ids) == oid).all()
    tol = (2 * span(zf, oid) * (score == R.SOFTMAX) + 64) * U * np.abs(ow) + 1e-36
    assert (np.abs(host(w) - ow) <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows_and_untouched_neighbours(dtype):
    T, E, k, ld = 37, 40, 4, 56
    wide = draw(T, E, dtype, 5, width=ld)
    z = wide[:, 8:8 + E]
    ids, w = run(z, T, E, k, R.SOFTMAX, None, True, 1.0, ldl=ld)
    oid, ow = R.router_topk(z.float().cpu().numpy(), k, R.SOFTMAX, None, True)
    assert (host(ids) == oid).all() and np.allclose(host(w), ow, rtol=2e-5, atol=1e-36)
    wide_d = torch.full((T, ld), 3.0, dtype=z.dtype, device="cuda")
    dz = wide_d[:, 8:8 + E]
    dw = np.random.default_rng(1).standard_normal((T, k)).astype(np.float32)
    dt = m.MOE_BF16 if dtype == "bf16" else m.MOE_F32
    m.moe_router_topk_backward(z, dt, ld, ids, dev_f32(dw), T, E, k, R.SOFTMAX, 1, 1.0, dz, ld)
    assert (wide_d[:, :8] == 3).all() and (wide_d[:, 8 + E:] == 3).all()
    o, mag = R.router_topk_backward(z.float().cpu().numpy(), oid, dw, R.SOFTMAX, True)
    assert (np.abs(dz.float().cpu().numpy() - o) <= 1e-4 * mag + 2.0 ** -8 * np.abs(o) + 1e-36).all()


def test_nan_logits_are_left_out_and_zero_rows_return():
    z = torch.tensor([[1.0, float("nan"), 0.5, 2.0], [float("nan")] * 4], device="cuda")
    ids, w = run(z, 2, 4, 3, R.SOFTMAX, None, False, 1.0)
    assert host(ids).tolist() == [[3, 0, 2], [0, 1, 2]]
    assert (host(w)[1] == 0).all() and np.isclose(host(w)[0].sum(), 1.0)
    empty = torch.empty(0, 4, device="cuda")
    ids, w = run(empty, 0, 4, 3, R.SOFTMAX, None, False, 1.0)
    assert ids.numel() == 0


BWD = [(1, 256, 8, "f32", R.SIGMOID, True, 2.5), (5, 13, 3, "bf16", R.SOFTMAX, False, 1.0), (130, 64, 8, "f32", R.SOFTMAX, True, 1.0),
       (67, 8, 8, "bf16", R.SIGMOID, True, 1.5), (9, 1024, 64, "f32", R.SOFTMAX, False, 1.0), (257, 72, 6, "bf16", R.SIGMOID, False, 2.5),
       (300, 256, 8, "bf16", R.SOFTMAX, True, 1.0), (1, 1, 1, "f32", R.SOFTMAX, False, 1.0), (17, 513, 2, "f32", R.SIGMOID, True, 1.0)]


@pytest.mark.parametrize("case", BWD, ids=str)
def test_backward_matches_the_oracle(case):
    T, E, k, dtype, score, renorm, scale = case
    z = draw(T, E, dtype, E + T)
    ids, _ = run(z, T, E, k, score, None, renorm, scale)
    ids = host(ids).copy()
    if T > 3 and k > 1:
        ids[0, 1] = ids[0, 0]                    # the same expert twice
        ids[3, 0] = E                            # out of range: takes no part
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    dz = torch.full((T, E), float("nan"), dtype=z.dtype, device="cuda")
    m.moe_router_topk_backward(z, m.MOE_BF16 if dtype == "bf16" else m.MOE_F32, E, dev_i32(ids), dev_f32(dw), T, E, k, score,
                               int(renorm), scale, dz, E)
    zf = z.float().cpu().numpy().astype(np.float64)
    rows = np.arange(T) != 3 if T > 3 and k > 1 else np.arange(T) >= 0
    o, mag = R.router_topk_backward(zf[rows], ids[rows], dw[rows], score, renorm, scale)
    D = span(zf[rows], ids[rows]).max(-1, keepdims=True) * (score == R.SOFTMAX)
    tol = (4 * D + 160) * U * mag + (2.0 ** -8 * np.abs(o) if dtype == "bf16" else 0) + 1e-36
    got = dz.float().cpu().numpy()
    assert (np.abs(got[rows] - o) <= tol).all()
    assert np.isfinite(got).all()
    assert (got[np.isneginf(zf)] == 0).all()


def test_backward_against_differences():
    """The float32 forward's own differences at a step where they mean something: weights move by w' h, their
    rounding is u, so a quotient over 2 h = 2^-5 is off by 2^-24 / 2^-5 and by h^2 / 6 of a third derivative
    below 1: 2^-10 together with the truncation."""
    T, E, k = 6, 24, 4
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(3)).cuda()
    for score in (R.SOFTMAX, R.SIGMOID):
        for renorm in (0, 1):
            ids, _ = run(z, T, E, k, score, None, renorm, 1.0)
            dw = torch.randn(T, k, generator=torch.Generator().manual_seed(4)).cuda()
            dz = torch.empty_like(z)
            m.moe_router_topk_backward(z, m.MOE_F32, E, ids, dw, T, E, k, score, renorm, 1.0, dz, E)
            base = host(ids)
            h = 2.0 ** -6
            for e in range(E):
                f = []
                for sgn in (1, -1):
                    zp = host(z).astype(np.float64)
                    zp[:, e] += sgn * h
                    f.append((R.weights_of(zp, base, score, renorm, 1.0) * host(dw)).sum(-1))
                num = (f[0] - f[1]) / (2 * h)
                assert np.abs(num - host(dz)[:, e]).max() < 2.0 ** -10


def test_other_stream_and_graph():
    T, E, k = 100, 64, 8
    z = draw(T, E, "f32", 77)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    dw, dz = torch.ones(T, k, device="cuda"), torch.empty_like(z)

    def step():
        m.moe_router_topk(z, m.MOE_F32, E, T, E, k, R.SOFTMAX, None, 1, 1.0, ids, w)
        m.moe_router_topk_backward(z, m.MOE_F32, E, ids, dw, T, E, k, R.SOFTMAX, 1, 1.0, dz, E)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(3):
        z.copy_(draw(T, E, "f32", seed))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [host(v).copy() for v in (ids, w, dz)]
        step()
        assert all(np.array_equal(a, host(b)) for a, b in zip(got, (ids, w, dz)))


def test_tensors_and_streams_of_another_device_are_refused(monkeypatch):
    z, ids, w = torch.zeros(2, 8, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, device="cuda")
    st = torch.cuda.Stream()
    args = (z, m.MOE_F32, 8, 2, 8, 2, R.SOFTMAX, None, 1, 1.0, ids, w)
    m.moe_router_topk(*args, stream=st)
    torch.cuda.synchronize()
    monkeypatch.setattr(m, "_current_device", lambda: z.get_device() + 1)
    for stream in (None, st):
        with pytest.raises(ValueError):
            m.moe_router_topk(*args, stream=stream)
    with pytest.raises(ValueError):
        m._stream_here(st)
    with pytest.raises(ValueError):
        m.moe_quantize_weights_mx4(torch.zeros(1, 32, 16, dtype=torch.bfloat16, device="cuda"), 1, 32, 16,
                                   torch.zeros(1, 16, 16, dtype=torch.uint8, device="cuda"), torch.zeros(1, 16, 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T,E,k,dtype,ldl,ldd", [(40, 100, 33, "f32", 100, 104), (19, 64, 64, "bf16", 67, 64), (21, 128, 17, "bf16", 132, 136),
                                                (18, 127, 16, "f32", 130, 127), (35, 4, 4, "f32", 8, 4)])
def test_backward_of_few_experts_many_choices_and_strides(T, E, k, dtype, ldl, ldd):
    z = draw(T, E, dtype, T, width=ldl)
    ids, _ = run(z, T, E, k, R.SIGMOID, None, False, 1.0, ldl=ldl)
    dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    zf = z.float().cpu().numpy()[:, :E]
    for score in (R.SOFTMAX, R.SIGMOID):
        for renorm in (False, True):
            dz = torch.full((T, ldd), 9.0, dtype=z.dtype, device="cuda")
            m.moe_router_topk_backward(z, m.MOE_BF16 if dtype == "bf16" else m.MOE_F32, ldl, ids, dev_f32(dw), T, E, k, score, int(renorm), 1.5,
                                       dz, ldd)
            o, mag = R.router_topk_backward(zf, host(ids), dw, score, renorm, 1.5)
            got = dz.float().cpu().numpy().astype(np.float64)
            D = np.maximum(span(zf, np.tile(np.arange(E), (T, 1))).max(-1), 0.0)[:, None]
            lim = (4 * D + 160) * U * mag
            assert (np.abs(got[:, :E] - o) <= lim + (2.0 ** -8 * (np.abs(o) + lim) if dtype == "bf16" else 0.0) + 1e-36).all(), (score, renorm)
            assert (got[:, E:] == 9).all()


def test_ids_stay_valid_without_finite_keys():
    """Outside what is supported: a bias that is not finite, logits of +inf.  The choice is unspecified, its ids are not."""
    E, k, T = 70, 8, 6
    z = draw(T, E, "f32", 1)
    z[1, ::3] = float("inf")
    bits = np.full(E, 0xFFFFFFFF, np.uint32)
    bits[1::4] = 0x7FC00000
    bits[2::4] = 0xFF800000
    for bias in (None, dev_f32(bits.view(np.float32))):
        for score in (R.SOFTMAX, R.SIGMOID):
            ids, _ = run(z, T, E, k, score, bias, True, 1.0)
            for row in host(ids):
                assert len(set(row.tolist())) == k and (row >= 0).all() and (row < E).all()


# ------------------------------------- gradients of weights that were left out
@pytest.mark.parametrize("E", [16, 96, 200])
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gradients_of_masked_slots_take_no_part(E, score, renorm):
    """A padded token's row, and slots whose expert was taken out: NaN and infinities there reach nothing."""
    T, k = 21, 4
    rng = np.random.default_rng([E, score, renorm])
    z = rng.standard_normal((T, E)).astype(np.float32)
    z[2::5] = -np.inf                                    # padded tokens
    z[3::5, 2:] = -np.inf                                # two experts left for four slots
    z[4, :] = np.nan
    zd = torch.from_numpy(z).cuda()
    ids, _ = run(zd, T, E, k, score, None, renorm, 1.0)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    masked = ~np.isfinite(np.take_along_axis(z, host(ids).astype(np.int64), -1))
    got = []
    for fill in ((0.0,), (np.nan, np.inf, -np.inf)):
        d = dw.copy()
        d[masked] = np.resize(np.array(fill, np.float32), masked.sum())
        dz = torch.full_like(zd, float("nan"))
        m.moe_router_topk_backward(zd, m.MOE_F32, E, ids, dev_f32(d), T, E, k, score, renorm, 1.0, dz, E)
        got.append(host(dz))
    assert masked.sum() > 10 and np.isfinite(got[0]).all() and np.array_equal(got[0], got[1])
    assert (got[1][~np.isfinite(z)] == 0).all()


# ------------------------------------------------------- logits far below zero
LOW = [(9, 5, 3, -95.0, 4.0), (33, 64, 8, -150.0, 30.0), (18, 127, 16, -60.0, 40.0), (17, 256, 8, -250.0, 20.0), (5, 200, 4, -80.0, 12.0)]


@pytest.mark.parametrize("T,E,k,mean,spread", LOW)
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_sigmoids_of_logits_far_below_zero(T, E, k, mean, spread, scale):
    """Scores below float32's range still have a ratio: renormalised weights sum to the factor, and their gradient is
    that of the ratio.  Tolerances as above: exponents of exact differences.  The oracle's own: it forms 1 - s from a
    float64 s.  For z <= 0 that is off by 2^-53 of itself; for z > 0, s lies in [1/2, 1) and is off by 2^-54, so 1 - s
    is off by 2^-54 in absolute terms, which every |g_j| carries twice at most (the diagonal and the renormalisation,
    whose factors s / S are at most 1 where S >= s >= 1/2): 2^-52 of the gradients' sum in rows with such a logit."""
    rng = np.random.default_rng([T, E])
    z = (mean + spread * rng.standard_normal((T, E))).astype(np.float32)
    z[0, : E // 2] = -np.inf
    if T > 8:
        z[3], z[4] = -np.inf, np.linspace(-20.0, -330.0, E).astype(np.float32)
        z[5, ::2] += 60.0
    zd = torch.from_numpy(z).cuda()
    for bias in (None, (0.1 * rng.standard_normal(E)).astype(np.float32)):
        for renorm in (False, True):
            ids, w = run(zd, T, E, k, R.SIGMOID, None if bias is None else dev_f32(bias), renorm, scale)
            oid, ow = R.router_topk(z, k, R.SIGMOID, bias, renorm, scale)
            assert (host(ids) == oid).all()
            assert (np.abs(host(w) - ow) <= 64 * U * np.abs(ow) + 1e-36).all(), (bias is None, renorm)
            alive = np.isfinite(np.take_along_axis(z, oid.astype(np.int64), -1)).any(-1)
            if renorm:
                assert np.allclose(host(w)[alive].sum(-1), scale, rtol=1e-5) and (host(w)[~alive] == 0).all()
            dw = rng.standard_normal((T, k)).astype(np.float32)
            dz = torch.full_like(zd, float("nan"))
            m.moe_router_topk_backward(zd, m.MOE_F32, E, ids, dev_f32(dw), T, E, k, R.SIGMOID, int(renorm), scale, dz, E)
            o, mag = R.router_topk_backward(z, oid, dw, R.SIGMOID, renorm, scale)
            above = (np.take_along_axis(z, oid.astype(np.int64), -1) > 0).any(-1, keepdims=True)
            own = above * 2.0 ** -52 * np.abs(dw * scale).sum(-1, keepdims=True)
            assert (np.abs(host(dz) - o) <= 160 * U * mag + own + 1e-36).all(), (bias is None, renorm)


# ----------------------------------------------------------------- many tokens
@pytest.mark.parametrize("E", [2, 130])
def test_more_tokens_than_one_launch_takes(E):
    """2^32 threads are the most a launch has: a wave a token, 2^26 of them."""
    T = (1 << 26) + 5 if E == 2 else (1 << 26) + 1
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    z[:, 1] = 1.0
    z[::7, 1] = -1.0
    z[:, 2:] = -4.0
    ids, w = torch.full((T, 1), -7, dtype=torch.int32, device="cuda"), torch.zeros(T, 1, device="cuda")
    m.moe_router_topk(z, m.MOE_BF16, E, T, E, 1, R.SIGMOID, None, 0, 1.0, ids, w)
    assert torch.equal(ids[:, 0], (z[:, 1] > 0).to(torch.int32))
    p = torch.sigmoid(torch.tensor([0.0, 1.0], dtype=torch.float64)).tolist()
    assert (w[ids == 0] - p[0]).abs().max().item() <= 64 * U and (w[ids == 1] - p[1]).abs().max().item() <= 64 * U
    dz = torch.full_like(z, 3.0)
    m.moe_router_topk_backward(z, m.MOE_BF16, E, ids, torch.ones_like(w), T, E, 1, R.SIGMOID, 0, 1.0, dz, E)
    d = [v * (1 - v) for v in p]
    for t in (0, 1, 7, (1 << 26) - 1, 1 << 26, T - 1):
        e = int(ids[t, 0])
        want = torch.zeros(E)
        want[e] = d[e]
        assert (dz[t].float().cpu() - want).abs().max().item() <= 2.0 ** -8 * d[e], t
    assert int((dz != 0).sum()) == T
