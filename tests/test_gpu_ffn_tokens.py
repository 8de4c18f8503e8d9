"""GPU parity of the few-token layer against the oracle.  The tolerance is
the oracle's: 1e-5 of every sum's magnitudes (tests/parity.py's rule 2)
carried through the activation and the second product, the hidden value's own
2^-16, and half a step of the output's type (bf16 2^-8, f32 2^-24)."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from oracle import mx4
from oracle.codec import e4m3_decode
from oracle.ffn_tokens import ffn_tokens
from oracle.quantize import quantize_weights
from tests.parity import dev_bf16, dev_f32, dev_i32, dev_u8, host
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu


class Layer:
    """Weights of El local experts: [2I, H] and [H, I] each, on the device and as values."""

    def __init__(self, fmt, El, H, I, seed=0, kb=(1, 1), nb=None):
        rng = np.random.default_rng([seed, H, I])
        self.fmt, self.El, self.H, self.I = fmt, El, H, I
        w01 = to_bf16_bits((rng.standard_normal((El, H, 2 * I)) * 0.05).astype(np.float32))
        wo = to_bf16_bits((rng.standard_normal((El, I, H)) * 0.05).astype(np.float32))
        self.v, self.q, self.s, self.blocks = [], [], [], []
        for w, K, N, b in ((w01, H, 2 * I, 0), (wo, I, H, 1)):
            if fmt == m.MOE_MX4:
                q, s = mx4.quantize_weights_mx4(w)
                self.v.append(mx4.decode(q, s))
                self.s.append(dev_u8(s))
                self.blocks += [0, 0]
            else:
                kbi, nbi = kb[b], (N, N)[b] if nb is None else nb[b]
                qk, s = quantize_weights(w, kbi, nbi)
                q = np.ascontiguousarray(qk.transpose(0, 2, 1))
                sv = np.repeat(np.repeat(s[:, :, 0, :].astype(np.float64), K // kbi, 1), N // nbi, 2)
                self.v.append(e4m3_decode(q) * sv.transpose(0, 2, 1))
                self.s.append(dev_f32(s))
                self.blocks += [kbi, nbi]
            self.q.append(dev_u8(q))

    def call(self, x, ldx, ids, tw, T, k, E, g0, dtype, out, ws, El=None):
        b = self.blocks
        m.moe_ffn_tokens(x, ldx, ids, tw, T, k, self.H, self.I, E, g0, self.El if El is None else El, self.fmt, self.q[0], self.s[0],
                         b[0], b[1], self.q[1], self.s[1], b[2], b[3], dtype, out, ws)

    def ws(self, T, k, E):
        return m.workspace(m.MOE_OP_FFN_TOKENS, T * k, self.H, self.I, E)


def routing(rng, T, k, E):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    return ids, rng.random((T, k)).astype(np.float32)


def check(got, o, tol, half):
    err = np.abs(got.astype(np.float64) - o)
    lim = tol + half * (np.abs(o) + tol) + 1e-36
    assert (err <= lim).all(), f"{(err > lim).sum()} of {err.size}, worst excess {(err - lim).max():.3g}"


CASES = [  # format, T, k, E, g0, El, H, I, kb, nb
    ("mx4", 1, 1, 1, 0, 1, 32, 32, None, None),
    ("mx4", 1, 8, 32, 0, 32, 512, 256, None, None),
    ("mx4", 7, 2, 8, 0, 8, 544, 96, None, None),
    ("mx4", 16, 4, 16, 4, 8, 256, 352, None, None),
    ("mx4", 64, 8, 8, 0, 8, 128, 160, None, None),
    ("e4m3", 1, 1, 1, 0, 1, 16, 16, (1, 1), None),
    ("e4m3", 1, 8, 32, 0, 32, 512, 256, (1, 1), None),
    ("e4m3", 2, 4, 16, 2, 9, 528, 272, (1, 1), None),
    ("e4m3", 17, 2, 4, 0, 4, 144, 80, (1, 1), (1, 1)),
    ("e4m3", 33, 1, 4, 0, 4, 256, 128, (2, 1), (2, 2)),
    ("e4m3", 40, 8, 16, 0, 16, 256, 384, (2, 3), None),
    ("e4m3", 64, 8, 64, 0, 64, 384, 256, (3, 2), (4, 3)),
    ("e4m3", 64, 16, 16, 0, 16, 256, 128, (1, 1), None),
    ("e4m3", 5, 3, 12, 3, 6, 1024, 1056, (1, 1), None),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_matches_the_oracle(case):
    fmt, T, k, E, g0, El, H, I, kb, nb = case
    L = Layer(m.MOE_MX4 if fmt == "mx4" else m.MOE_E4M3FN, El, H, I, seed=T, kb=kb, nb=nb)
    rng = np.random.default_rng([T, k, E, H])
    ids, tw = routing(rng, T, k, E)
    xb = to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    o, tol = ffn_tokens(xb, ids, tw, L.v[0], L.v[1], g0, El, E)
    ws = L.ws(T, k, E)
    print("ffn_tokens", case, flush=True)
    for dtype, tt, half in ((m.MOE_F32, torch.float32, 2.0 ** -24), (m.MOE_BF16, torch.bfloat16, 2.0 ** -8)):
        out = torch.full((T, H), 7.0, dtype=tt, device="cuda")
        L.call(dev_bf16(xb), H, dev_i32(ids), dev_f32(tw), T, k, E, g0, dtype, out, ws)
        assert m.moe_debug_check(ws) == 0
        check(out.float().cpu().numpy(), o, tol, half)
        again = torch.empty_like(out)
        L.call(dev_bf16(xb), H, dev_i32(ids), dev_f32(tw), T, k, E, g0, dtype, again, ws)
        assert torch.equal(out.view(torch.uint8), again.view(torch.uint8)), "the same call gives the same bits"


@pytest.mark.parametrize("fmt", [m.MOE_MX4, m.MOE_E4M3FN])
def test_repeated_experts_bad_ids_and_tokens_without_an_expert(fmt):
    T, k, E, g0, El, H, I = 24, 4, 16, 4, 6, 288, 160
    L = Layer(fmt, El, H, I)
    rng = np.random.default_rng(9)
    ids, tw = routing(rng, T, k, E)
    ids[0] = 5                                          # the same expert four times
    ids[1:20, 0] = 6                                    # more than one block of rows for one expert
    ids[3] = [0, 1, 2, 3]                               # no local expert: zeros
    ids[4] = [-1, E, 2 ** 31 - 1, -2 ** 31]             # not experts at all
    xb = to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    o, tol = ffn_tokens(xb, ids, tw, L.v[0], L.v[1], g0, El, E)
    ws = L.ws(T, k, E)
    wide = torch.zeros(T, H + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + H] = dev_bf16(xb)
    out = torch.full((T, H), 7.0, device="cuda")
    L.call(wide[:, 8:8 + H], H + 24, dev_i32(ids), dev_f32(tw), T, k, E, g0, m.MOE_F32, out, ws)
    check(host(out), o, tol, 2.0 ** -24)
    assert (host(out)[3:5] == 0).all()
    assert m.moe_debug_check(ws) == m.MOE_DEVERR_EXPERT_ID
    # no local expert at all: zeros, the weights are not looked at
    out.fill_(7.0)
    ws = L.ws(T, k, E)
    L.call(dev_bf16(xb), H, dev_i32(np.minimum(ids, 3).clip(0)), dev_f32(tw), T, k, E, g0, m.MOE_F32, out, ws)
    assert (host(out) == 0).all() and m.moe_debug_check(ws) == 0
    out.fill_(7.0)
    L.call(dev_bf16(xb), H, dev_i32(ids.clip(0, E - 1)), dev_f32(tw), T, k, E, g0, m.MOE_F32, out, ws, El=0)
    assert (host(out) == 0).all()


@pytest.mark.parametrize("fmt", [m.MOE_MX4, m.MOE_E4M3FN])
def test_a_bad_token_stays_its_own(fmt):
    T, k, E, H, I = 19, 2, 4, 256, 128
    L = Layer(fmt, E, H, I)
    rng = np.random.default_rng(2)
    ids, tw = routing(rng, T, k, E)
    xb = to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    clean = torch.empty(T, H, device="cuda")
    ws = L.ws(T, k, E)
    L.call(dev_bf16(xb), H, dev_i32(ids), dev_f32(tw), T, k, E, 0, m.MOE_F32, clean, ws)
    xb[5, 17], xb[9, 200] = 0x7FC0, 0x7F80              # NaN, infinity
    out = torch.empty(T, H, device="cuda")
    L.call(dev_bf16(xb), H, dev_i32(ids), dev_f32(tw), T, k, E, 0, m.MOE_F32, out, ws)
    keep = np.ones(T, bool)
    keep[[5, 9]] = False
    assert np.array_equal(host(out)[keep], host(clean)[keep])
    assert np.isnan(host(out)[5]).all() and not np.isfinite(host(out)[9]).any()


def test_a_token_does_not_depend_on_the_batch():
    """Alone, or with others at its expert: the same bits."""
    E, k, H, I = 8, 2, 512, 256
    for fmt in (m.MOE_MX4, m.MOE_E4M3FN):
        L = Layer(fmt, E, H, I)
        rng = np.random.default_rng(6)
        ids, tw = routing(rng, 40, k, E)
        xb = to_bf16_bits(rng.standard_normal((40, H)).astype(np.float32))
        ws = L.ws(64, k, E)
        out = torch.empty(40, H, device="cuda")
        L.call(dev_bf16(xb), H, dev_i32(ids), dev_f32(tw), 40, k, E, 0, m.MOE_F32, out, ws)
        one = torch.empty(1, H, device="cuda")
        for t in (0, 13, 39):
            L.call(dev_bf16(xb[t:t + 1]), H, dev_i32(ids[t:t + 1]), dev_f32(tw[t:t + 1]), 1, k, E, 0, m.MOE_F32, one, ws)
            assert np.array_equal(host(one)[0], host(out)[t])


def test_streams_graph_replays_and_a_shared_workspace():
    T, k, E, H, I = 12, 4, 16, 512, 256
    A, B = Layer(m.MOE_MX4, E, H, I, seed=1), Layer(m.MOE_E4M3FN, E, H, I, seed=2)
    rng = np.random.default_rng(3)
    ids, tw = routing(rng, T, k, E)
    x = dev_bf16(to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32)))
    di, dw = dev_i32(ids), dev_f32(tw)
    ws = A.ws(T, k, E)
    mid, out = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():                                          # two layers, one workspace, in order
        A.call(x, H, di, dw, T, k, E, 0, m.MOE_BF16, mid, ws)
        B.call(mid, H, di, dw, T, k, E, 0, m.MOE_BF16, out, ws)

    step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for r in range(4):
        ids, tw = routing(rng, T, k, E)
        di.copy_(dev_i32(ids))
        x.copy_(dev_bf16(to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [host(v).copy() for v in (mid, out)]
        step()
        assert all(np.array_equal(a, host(b)) for a, b in zip(got, (mid, out)))
    assert m.moe_debug_check(ws) == 0


LONG = [  # rows and weights beyond what a workgroup stages or takes at once
    ("mx4", 20, 2, 2, 0, 2, 2336, 1120, None, None),          # 20 slots an expert, both contractions in parts, short last chunks
    ("e4m3", 20, 2, 2, 0, 2, 2352, 1040, (1, 1), None),
    ("e4m3", 3, 4, 8, 0, 8, 48, 4112, (1, 1), None),          # several units a wave, some left over
    ("mx4", 5, 8, 8, 0, 8, 8224, 64, None, None),             # the first contraction in parts, many output columns
    ("e4m3", 17, 4, 4, 0, 4, 2080, 4112, (1, 1), None),       # parts, passes and a wave's own units together
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_rows_and_many_units(case):
    test_matches_the_oracle(case)


@pytest.mark.parametrize("fmt", [m.MOE_MX4, m.MOE_E4M3FN])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_token_alone_and_in_a_batch_of_many_units(fmt, dtype):
    """The batch gives every workgroup more than four units of an expert, the token alone one or two: units that a wave
    forms by itself and units that four waves share."""
    E, H, I, T = 16, 2560, 1600, 64
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, s, blocks = [], [], []
    for N, K in ((2 * I, H), (H, I)):
        if fmt == m.MOE_MX4:
            q.append(torch.randint(0, 256, (E, N, K // 2), generator=gen, dtype=torch.uint8, device="cuda"))
            s.append(torch.randint(118, 122, (E, N, K // 32), generator=gen, dtype=torch.uint8, device="cuda"))
            blocks += [0, 0]
        else:
            q.append((torch.randn(E, N, K, generator=gen, device="cuda") * 0.5).to(torch.float8_e4m3fn).view(torch.uint8))
            s.append(torch.rand(E, 1, 1, N, generator=gen, device="cuda") * 0.1)
            blocks += [1, N]
    x = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
    ws = m.workspace(m.MOE_OP_FFN_TOKENS, T * 2, H, I, E)
    # experts by chance, and all tokens at two of them: passes of 16 slots, whose rows are staged by parts
    for k, met in ((1, E), (2, E), (2, 2)):
        ids = torch.rand(T, met, generator=gen, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
        tw = torch.rand(T, k, generator=gen, device="cuda")

        def call(rows):
            n = len(rows)
            out = torch.empty(n, H, dtype=dtype, device="cuda")
            m.moe_ffn_tokens(x[rows].contiguous(), H, ids[rows].contiguous(), tw[rows].contiguous(), n, k, H, I, E, 0, E, fmt, q[0], s[0],
                             blocks[0], blocks[1], q[1], s[1], blocks[2], blocks[3], m.MOE_F32 if dtype == torch.float32 else m.MOE_BF16, out, ws)
            return out
        batch = call(list(range(T)))
        assert torch.isfinite(batch).all()
        for rows in ([0], [31], [63], [5, 9], list(range(20, 33))):
            assert torch.equal(call(rows), batch[rows]), (k, rows)


@pytest.mark.parametrize("T", [1, 21])
def test_weights_without_a_value_reach_their_own_results_only(T):
    """Scale 255 (what the quantizer writes, with codes 0, for a block that is not finite) in one block."""
    E, k, H, I = 4, 2, 288, 160
    L = Layer(m.MOE_MX4, E, H, I, seed=T)
    rng = np.random.default_rng([T, 5])
    ids, tw = routing(rng, T, k, E)
    ids[0] = [2, 1]
    xb = to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    xb[:, 64:96] = 0                                     # zeros at the block too: zero times NaN is NaN
    out, ws = torch.empty(T, H, device="cuda"), L.ws(T, k, E)

    def call():
        L.call(dev_bf16(xb), H, dev_i32(ids), dev_f32(tw), T, k, E, 0, m.MOE_F32, out, ws)
        return host(out).copy()
    clean = call()
    meets = (ids == 2).any(1)
    for row in (17, I + 17):                             # a gate row, an up row: the whole token
        q, s = L.q[0].clone(), L.s[0].clone()
        L.q[0][2, row, 32:48], L.s[0][2, row, 2] = 0, 255
        got = call()
        assert np.isnan(got[meets]).all() and np.array_equal(got[~meets], clean[~meets])
        L.q[0].copy_(q), L.s[0].copy_(s)
    L.q[1][2, 100, 64:80], L.s[1][2, 100, 4] = 0, 255    # an output channel
    got = call()
    bad = np.zeros((T, H), bool)
    bad[meets, 100] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


def test_smallest_and_largest_scales():
    """Scale codes 0 (2^-127, below the normal range) and 252, the largest that a quantizer writes."""
    T, k, E, H, I = 3, 1, 1, 64, 32
    L = Layer(m.MOE_MX4, E, H, I, seed=3)
    rng = np.random.default_rng(4)
    ids = np.zeros((T, k), np.int32)
    for up, down, xs, w in ((0, 127, 2.0 ** 122, 1.0), (252, 127, 2.0 ** -124, 1.0), (127, 0, 2.0 ** -4, 2.0 ** 120), (127, 252, 2.0 ** -10, 2.0 ** -120)):
        q = [rng.integers(0, 256, tuple(v.shape), dtype=np.uint8) for v in L.q]
        s = [np.full(tuple(v.shape), c, np.uint8) for v, c in zip(L.s, (up, down))]
        L.q, L.s = [dev_u8(v) for v in q], [dev_u8(v) for v in s]
        xb = to_bf16_bits((rng.standard_normal((T, H)) * xs).astype(np.float32))
        tw = np.full((T, k), w, np.float32)
        o, tol = ffn_tokens(xb, ids, tw, mx4.decode(q[0], s[0]), mx4.decode(q[1], s[1]), 0, E, E)
        out, ws = torch.empty(T, H, device="cuda"), L.ws(T, k, E)
        L.call(dev_bf16(xb), H, dev_i32(ids), dev_f32(tw), T, k, E, 0, m.MOE_F32, out, ws)
        assert np.abs(o).max() > 1e-6
        # a slot's own result near 2^-127 is held to 2^-149, the step of float32 there
        check(host(out), o, tol + w * 2.0 ** -148, 2.0 ** -24)
