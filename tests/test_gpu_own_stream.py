"""Every call of the router, the 4-bit format and the few-token layer runs on
the stream it is given, or on the current one: its outputs are poisoned, the
default stream is kept busy, and the results are there, read on that stream
alone, while the default stream is still at work."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from tests.parity import host

pytestmark = pytest.mark.gpu
T, E, k, H, I = 96, 16, 4, 256, 128


def gen():
    return torch.Generator(device="cuda").manual_seed(3)


def router(o, s):
    z = torch.randn(T, E, generator=gen(), device="cuda")
    dw = torch.randn(T, k, generator=gen(), device="cuda")

    def call():
        m.moe_router_topk(z, m.MOE_F32, E, T, E, k, m.MOE_SCORE_SOFTMAX, None, 1, 1.0, o["ids"], o["w"], **s)
        m.moe_router_topk_backward(z, m.MOE_F32, E, o["ids"], dw, T, E, k, m.MOE_SCORE_SOFTMAX, 1, 1.0, o["dz"], E, **s)
    return call


def format4(o, s):
    x = torch.randn(T, H, generator=gen(), device="cuda").to(torch.bfloat16)
    w = torch.randn(E, H, I, generator=gen(), device="cuda").to(torch.bfloat16)

    def call():
        m.moe_quantize_rows_mx4(x, None, H, m.MOE_ACT_NONE, T, H, o["q"], H // 2, o["s"], H // 32, **s)
        m.moe_quantize_weights_mx4(w, E, H, I, o["wq"], o["ws"], **s)
        m.moe_dequantize_rows_mx4(o["q"], H // 2, o["s"], H // 32, T, H, m.MOE_F32, o["x"], H, **s)
    return call


def product(o, s):
    u8 = dict(generator=gen(), dtype=torch.uint8, device="cuda")
    q, qs = torch.randint(0, 256, (T, H // 2), **u8), torch.randint(120, 128, (T, H // 32 + 1), **u8)     # scales copied first
    w, ws = torch.randint(0, 256, (E, I, H // 2), **u8), torch.randint(120, 128, (E, I, H // 32), **u8)
    sizes, work = torch.full((E,), T // E, dtype=torch.int32, device="cuda"), m.workspace(m.MOE_OP_GMM_MX4, T, H, I, E)

    def call():
        m.moe_gmm_mx4(q, H // 2, qs[:, :H // 32], H // 32 + 1, m.MOE_MX4, 0, w, ws, sizes, E, 0, E, T, H, I, m.MOE_F32, o["y"], work, **s)
    return call


def layer(o, s):
    u8, n = dict(generator=gen(), dtype=torch.uint8, device="cuda"), 16
    w01, s01 = torch.randint(0, 256, (E, 2 * I, H // 2), **u8), torch.randint(118, 122, (E, 2 * I, H // 32), **u8)
    wo, so = torch.randint(0, 256, (E, H, I // 2), **u8), torch.randint(118, 122, (E, H, I // 32), **u8)
    x = torch.randn(n, H, generator=gen(), device="cuda").to(torch.bfloat16)
    ids = torch.rand(n, E, generator=gen(), device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    tw, work = torch.rand(n, k, generator=gen(), device="cuda"), m.workspace(m.MOE_OP_FFN_TOKENS, n * k, H, I, E)

    def call():
        m.moe_ffn_tokens(x, H, ids, tw, n, k, H, I, E, 0, E, m.MOE_MX4, w01, s01, 0, 0, wo, so, 0, 0, m.MOE_F32, o["out"], work, **s)
    return call


def nan(*shape):
    return torch.full(shape, float("nan"), device="cuda")


def bytes_(*shape):
    return torch.full(shape, 0xAA, dtype=torch.uint8, device="cuda")


SETS = {
    "router": (router, lambda: dict(ids=torch.full((T, k), -7, dtype=torch.int32, device="cuda"), w=nan(T, k), dz=nan(T, E))),
    "format": (format4, lambda: dict(q=bytes_(T, H // 2), s=bytes_(T, H // 32), wq=bytes_(E, I, H // 2), ws=bytes_(E, I, H // 32), x=nan(T, H))),
    "product": (product, lambda: dict(y=nan(T, I))),
    "layer": (layer, lambda: dict(out=nan(16, H))),
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
