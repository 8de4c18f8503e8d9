"""Every call of the b128 format and of the balance loss runs on the stream it
is given, or on the current one: its outputs are poisoned, the default stream
is kept busy, and the results are there, read on that stream alone, while the
default stream is still at work.  And buffers that pass 2^32 bytes."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from oracle import b128
from oracle.codec import e4m3_decode
from tests.parity import dev_i32, host

pytestmark = pytest.mark.gpu
T, E, k, H, I = 96, 16, 4, 256, 128


def gen():
    return torch.Generator(device="cuda").manual_seed(3)


def bf(*shape):
    return torch.randn(*shape, generator=gen(), device="cuda").to(torch.bfloat16)


def u8(low, high, *shape):
    return torch.randint(low, high, shape, generator=gen(), dtype=torch.uint8, device="cuda")


def sizes():
    return torch.full((E,), T // E, dtype=torch.int32, device="cuda")


def quantizers(o, s):
    x, w, g, ws = bf(T, H), bf(E, H, I), sizes(), torch.zeros(256, dtype=torch.uint8, device="cuda")

    def call():
        m.moe_quantize_rows_b128(x, None, H, m.MOE_ACT_NONE, T, H, o["q"], H, o["s"], H // 128, **s)
        m.moe_quantize_weights_b128(w, E, H, I, o["wq"], o["ws"], o["wqt"], o["wst"], **s)
        m.moe_quantize_cols_b128(x, None, H, m.MOE_ACT_NONE, T, 1, None, g, E, 0, E, T, H, o["ct"], o["cs"], ws, **s)
    return call


def products(o, s):
    x, xs, w, ws = u8(0, 0x7F, T, H), u8(118, 122, T, 16), u8(0, 0x7F, E, I, H), u8(118, 122, E, H // 128, 1, I // 128)
    n = m.tgmm_xt_cols(T, E) // 128
    xt, xts, yt, yts = u8(0, 0x7F, n, H, 128), u8(118, 122, n, H), u8(0, 0x7F, n, I, 128), u8(118, 122, n, I)
    g, a, b = sizes(), m.workspace(m.MOE_OP_GMM_B128, T, H, I, E), m.workspace(m.MOE_OP_TGMM_B128, T, H, I, E)

    def call():
        m.moe_gmm_b128(x, H, xs[:, :H // 128], 16, w, ws, m.MOE_E8M0, g, E, 0, E, T, H, I, m.MOE_F32, o["y"], a, **s)
        m.moe_tgmm_b128(xt, xts, yt, yts, g, E, 0, E, T, H, I, m.MOE_F32, o["dw"], b, **s)
    return call


def balance(o, s):
    z = torch.randn(T, E, generator=gen(), device="cuda")
    ids = torch.rand(T, E, generator=gen(), device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    off, dl, ws = dev_i32([0, 50, T]), torch.ones(2, device="cuda"), m.workspace(m.MOE_OP_BALANCE, T, 2, 0, E)

    def call():
        m.moe_balance_loss(z, m.MOE_F32, E, ids, T, E, k, m.MOE_SCORE_SOFTMAX, off, 2, o["loss"], o["counts"], o["tokens"], ws, **s)
        m.moe_balance_loss_backward(z, m.MOE_F32, E, o["counts"], o["tokens"], dl, T, E, k, m.MOE_SCORE_SOFTMAX, off, 2, 0, o["dz"], E, **s)
    return call


def nan(*shape):
    return torch.full(shape, float("nan"), device="cuda")


def bytes_(*shape):
    return torch.full(shape, 0xAA, dtype=torch.uint8, device="cuda")


def ints(*shape):
    return torch.full(shape, -7, dtype=torch.int32, device="cuda")


SETS = {
    "quantizers": (quantizers, lambda: dict(q=bytes_(T, H), s=bytes_(T, H // 128), wq=bytes_(E, I, H), ws=bytes_(E, H // 128, 1, I // 128),
                                            wqt=bytes_(E, H, I), wst=bytes_(E, I // 128, 1, H // 128), ct=bytes_(m.tgmm_xt_cols(T, E) // 128, H, 128),
                                            cs=bytes_(m.tgmm_xt_cols(T, E) // 128, H))),
    "products": (products, lambda: dict(y=nan(T, I), dw=nan(E, H, I))),
    "balance": (balance, lambda: dict(loss=nan(2), counts=ints(2, E), tokens=ints(2), dz=nan(T, E))),
}


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("name", SETS)
def test_results_are_there_while_the_default_stream_is_busy(name, explicit):
    make, outputs = SETS[name]
    want, got, st = outputs(), outputs(), torch.cuda.Stream()
    first = {n: host(v).copy() for n, v in want.items()}
    make(want, {})()
    call = make(got, dict(stream=st) if explicit else {})
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)                       # a bounded spin of 0.1 to 0.3 s
    if explicit:
        call()
    with torch.cuda.stream(st):
        if not explicit:
            call()
        got = {n: host(v) for n, v in got.items()}       # copied, and waited for, on this stream
    assert not torch.cuda.default_stream().query(), "the default stream ended too early to tell"
    torch.cuda.synchronize()
    for n, v in want.items():
        assert np.array_equal(host(v), got[n]) and not np.array_equal(got[n], first[n]), n
        assert got[n].dtype != np.float32 or np.isfinite(got[n]).all(), n


# ------------------------------------------------------------ past 2^32 bytes
@pytest.mark.parametrize("narrow", [True, False])
def test_rows_far_apart(narrow):
    """Rows of codes and scales 2^22 bytes apart, 1100 of them: past 2^32 bytes, in the quantizer and in the product."""
    R, K, N, ld = 1100, 272, 144 if narrow else 256 * 256, 1 << 22
    x, w = bf(R, K), bf(1, K, N)
    far = torch.empty(R * ld, dtype=torch.uint8, device="cuda").view(R, ld)
    q, s = far[:, :K], far[:, K:K + 3]
    m.moe_quantize_rows_b128(x, None, K, m.MOE_ACT_NONE, R, K, q, ld, s, ld)
    oq, os_ = b128.quantize_rows_b128(host(x))
    assert np.array_equal(q.cpu().numpy(), oq) and np.array_equal(s.cpu().numpy(), os_)
    wq, ws = bytes_(1, N, K), bytes_(1, 3, 1, -(-N // 128))
    m.moe_quantize_weights_b128(w, 1, K, N, wq, ws, None, None)
    near = torch.zeros(R, 304, dtype=torch.uint8, device="cuda")
    m.moe_quantize_rows_b128(x, None, K, m.MOE_ACT_NONE, R, K, near, 304, near[:, K:K + 3], 304)
    out = [nan(R, N) for _ in range(2)]
    for a, l, o in ((far, ld, out[0]), (near, 304, out[1])):
        m.moe_gmm_b128(a[:, :K], l, a[:, K:K + 3], l, wq, ws, m.MOE_E8M0, dev_i32([R]), 1, 0, 1, R, K, N, m.MOE_F32, o,
                       m.workspace(m.MOE_OP_GMM_B128, R, K, N, 1))
    assert torch.equal(*out) and not torch.isnan(out[0]).any()


def test_weights_and_gradients_past_32_bits():
    """Two experts of 65536 by 36864: the second one's codes begin past 2^31 and end past 2^32 bytes, its gradient past 2^34."""
    E2, K, N, R = 2, 65536, 36864, 130
    w = torch.empty(E2, K, N, dtype=torch.bfloat16, device="cuda")
    w.fill_(0.5)
    w[1, -200:, -40:] = bf(200, 40)
    q, s = torch.empty(E2, N, K, dtype=torch.uint8, device="cuda"), bytes_(E2, K // 128, 1, N // 128)
    qt, st = torch.empty(E2, K, N, dtype=torch.uint8, device="cuda"), bytes_(E2, N // 128, 1, K // 128)
    m.moe_quantize_weights_b128(w, E2, K, N, q, s, qt, st)
    oq, os_ = b128.quantize_weights_b128(host(w[1:, -256:, -128:].contiguous()))
    assert np.array_equal(qt[1, -256:, -128:].cpu().numpy(), oq[0]) and np.array_equal(q[1, -128:, -256:].cpu().numpy(), oq[0].T)
    assert np.array_equal(s[1, -2:, 0, -1:].cpu().numpy(), os_[0]) and np.array_equal(st[1, -1:, 0, -2:].cpu().numpy(), os_[0].T)
    w_max = float(w[1, -256:, -128:].abs().max())
    del w, qt
    # the product: ones at the last inputs only
    gs, x, xs = dev_i32([1, R - 1]), torch.zeros(R, K, dtype=torch.uint8, device="cuda"), torch.full((R, K // 128), 127, dtype=torch.uint8, device="cuda")
    x[:, -256:] = 0x38
    out, ws = nan(R, N), m.workspace(m.MOE_OP_GMM_B128, R, K, N, E2)
    m.moe_gmm_b128(x, K, xs, K // 128, q, s, m.MOE_E8M0, gs, E2, 0, E2, R, K, N, m.MOE_F32, out, ws)
    want = (e4m3_decode(oq[0]) * np.repeat(b128.scale_values(os_[0]), 128, axis=0)).sum(axis=0)
    # 256 products with codes below 2^9 (exponent 8) and scales of 2^-6 at most (values below 7), each cut below 2^-12 of 2^8: 256 * 2^(8 - 6 - 12)
    assert np.abs(w_max) < 7 and np.abs(host(out)[-1, -128:] - want).max() <= 0.25 and (host(out)[0] == 128).all() and m.moe_debug_check(ws) == 0
    del q, out, x
    # the weight gradient: ones in the last rows and columns
    cols = m.tgmm_xt_cols(R, E2)
    a, b = (torch.zeros(cols // 128, C, 128, dtype=torch.uint8, device="cuda") for C in (K, N))
    for t, n in ((a, 3), (b, 5)):                        # 129 rows of the second expert: blocks 1 and 2
        t[1, -n:], t[2, -n:, :1] = 0x38, 0x38
    dw, ws = torch.full((E2, K, N), 7.0, device="cuda"), m.workspace(m.MOE_OP_TGMM_B128, R, K, N, E2)
    m.moe_tgmm_b128(a, torch.full((cols // 128, K), 127, dtype=torch.uint8, device="cuda"), b,
                    torch.full((cols // 128, N), 127, dtype=torch.uint8, device="cuda"), gs, E2, 0, E2, R, K, N, m.MOE_F32, dw, ws)
    assert (dw[1, -3:, -5:] == R - 1).all() and int(torch.count_nonzero(dw)) == 15 and m.moe_debug_check(ws) == 0


def test_columns_of_tokens_past_32_bits():
    """Tokens whose buffer passes 2^32 elements, gathered from its end."""
    C, ld, n, k2 = 144, (1 << 23) + 8, 600, 2
    far = torch.empty(n * ld, dtype=torch.bfloat16, device="cuda").view(n, ld)
    x = far[:, :C]
    x.copy_(bf(n, C))
    perm = torch.randperm(n * k2, generator=gen(), device="cuda").to(torch.int32)
    gs, M = [500, 0, 700], n * k2
    cols = m.tgmm_xt_cols(M, 3)
    qt, st, ws = bytes_(cols // 128, C, 128), bytes_(cols // 128, C), torch.zeros(256, dtype=torch.uint8, device="cuda")
    m.moe_quantize_cols_b128(x, None, ld, m.MOE_ACT_NONE, n, k2, perm, dev_i32(gs), 3, 0, 3, M, C, qt, st, ws)
    v = b128.values(host(x.contiguous())[host(perm) // k2])
    oq, os_, used = b128.quantize_cols_b128(v, np.array(gs), 0, 3, M, cols)
    assert np.array_equal(b128.columns_of(host(qt))[:, used], oq[:, used]) and np.array_equal(host(st)[used[::128]], os_[used[::128]])


def test_blocks_of_rows_past_32_bits():
    """1100 blocks of 128 rows of 32768 columns: codes past 2^32 bytes, in the quantizer and in the weight gradient."""
    n, C, N = 1100, 32768, 16
    M = 128 * n
    x = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    x[-128:] = bf(128, C)
    cols, gs = m.tgmm_xt_cols(M, 1), dev_i32([M])
    qt, st = torch.empty(cols // 128, C, 128, dtype=torch.uint8, device="cuda"), bytes_(cols // 128, C)
    ws = m.workspace(m.MOE_OP_TGMM_B128, M, C, N, 1)
    m.moe_quantize_cols_b128(x, None, C, m.MOE_ACT_NONE, M, 1, None, gs, 1, 0, 1, M, C, qt, st, ws)
    oq, os_, _ = b128.quantize_cols_b128(b128.values(host(x[-128:])), np.array([128]), 0, 1, 128, 128)
    assert np.array_equal(b128.columns_of(host(qt[n - 1:n])), oq) and np.array_equal(host(st[n - 1:n]), os_)
    assert not qt[:n - 1].any() and (st[:n - 1] == 127).all()
    y, ys = torch.zeros(cols // 128, N, 128, dtype=torch.uint8, device="cuda"), torch.full((cols // 128, N), 127, dtype=torch.uint8, device="cuda")
    y[n - 1, 3] = 0x38                                   # ones
    dw = nan(1, C, N)
    m.moe_tgmm_b128(qt, st, y, ys, gs, 1, 0, 1, M, C, N, m.MOE_F32, dw, ws)
    want = (e4m3_decode(oq) * b128.scale_values(os_).T).sum(axis=1)
    # 128 products with codes below 2^9 (exponent 8), each cut below 2^-12 of 2^8, and a float32 sum of 128 terms in chunks of 8
    lim = b128.scale_values(os_)[0] * (128 * 2.0 ** (8 - 12) + 32 * 2.0 ** -24 * 128 * 512)
    got = host(dw)[0]
    assert (np.abs(got[:, 3] - want) <= lim).all() and not np.delete(got, 3, axis=1).any() and m.moe_debug_check(ws) == 0
