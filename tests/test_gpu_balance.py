"""GPU parity of the balance loss and its gradient against the oracle.

Counts and tokens are equal.  Tolerances (u = 2^-24, derived as the router's):
a share is a score over a sum: expf within 4 u of a value whose argument
z - m was rounded once (|z - m| u, and at most 110 u where it counts), the
sum of up to 1024 of them 22 u, quotient and product 4 u: w = (2 D + 64) u
with D <= 32 here (logits within +-16; the lowest values have share 0).  The
loss adds up to 2^15 positive shares of a sequence in 32 bits, in runs of a
wave, four waves and the slots, each run at most 1024 long: 3 * 1024 u at most, and E
products: the sum of positive terms, relative (w + 4 * 1024 u).  The gradient: p (c - sum c p): (4 w + 64 u) of the
magnitudes' sum, half a bf16 step where it is bf16; added to a float32 value,
one rounding of the sum."""

import numpy as np
import pytest
import torch

import moe_fp8_grouped_amd as m
from oracle import balance as B
from tests.parity import dev_f32, dev_i32, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
W = (2 * 32 + 64) * U
NEG = float(np.finfo(np.float32).min)

CASES = [  # T, E, k, dtype, score, sequences' lengths (None: all rows, no offsets), rows in front and behind
    (1, 256, 8, "f32", B.SOFTMAX, None, 0, 0),
    (1, 1, 1, "bf16", B.SIGMOID, None, 0, 0),
    (5, 13, 3, "bf16", B.SOFTMAX, [0, 3, 1, 0], 1, 0),
    (130, 64, 8, "f32", B.SIGMOID, [64, 66], 0, 0),
    (300, 72, 6, "f32", B.SOFTMAX, [1] * 33 + [0, 31, 32, 97, 64], 10, 33),
    (33, 1024, 64, "f32", B.SOFTMAX, None, 0, 0),
    (257, 513, 1, "bf16", B.SIGMOID, [200, 57], 0, 0),
    (1000, 129, 4, "bf16", B.SOFTMAX, [500, 0, 0, 499], 0, 1),
    (5000, 256, 8, "bf16", B.SIGMOID, [4096, 3, 901], 0, 0),
    (33000, 8, 2, "f32", B.SOFTMAX, [20000, 12000], 500, 500),
    (4099, 128, 6, "f32", B.SIGMOID, [4099], 0, 0),
    (64, 40, 3, "f32", B.SOFTMAX, [0, 0, 0], 32, 32),
]


def draw(T, E, k, dtype, seed, width=None):
    """Logits with masked experts, rows without one (-inf, NaN or the type's lowest value), and far ones."""
    rng = np.random.default_rng(seed)
    z = np.clip(rng.standard_normal((T, width or E)) * 2 + rng.standard_normal(width or E), -16, 16).astype(np.float32)
    if T > 2:
        z[rng.random(z.shape) < 0.05] = -np.inf
        z[1::7] = -np.inf
        z[2::11] = NEG
        z[3::13] = np.nan
        z[0, ::2] = NEG
    t = torch.from_numpy(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    ids = rng.integers(0, E, (T, k)).astype(np.int32)       # any choice: taken-out experts and repeated ones among them
    if T > 4:
        ids[4, 0], ids[0, 0] = -1, E
    return t, ids


def offsets(lengths, front):
    return front + np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def forward(z, ids, E, k, score, off, ldl=None, ws=None):
    T, S = z.shape[0], 1 if off is None else len(off) - 1
    dt = m.MOE_BF16 if z.dtype == torch.bfloat16 else m.MOE_F32
    loss = torch.full((S,), float("nan"), device="cuda")
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.full((m.workspace_bytes(m.MOE_OP_BALANCE, T, S, 0, E),), 0xFF, dtype=torch.uint8, device="cuda")
        ws[:4] = 0                                          # all but the error word may hold anything
    m.moe_balance_loss(z, dt, ldl or E, dev_i32(ids), T, E, k, score, None if off is None else dev_i32(off), S, loss, counts,
                       tokens, ws)
    return loss, counts, tokens, ws


def backward(z, counts, tokens, dloss, E, k, score, off, acc=0, into=None, ldl=None, ldd=None):
    T, S = z.shape[0], tokens.shape[0]
    dt = m.MOE_BF16 if z.dtype == torch.bfloat16 else m.MOE_F32
    dz = torch.full_like(z, 9.0) if into is None else into
    m.moe_balance_loss_backward(z, dt, ldl or E, counts, tokens, dloss, T, E, k, score, None if off is None else dev_i32(off), S, acc,
                                dz, ldd or E)
    return dz


@pytest.mark.parametrize("case", CASES, ids=str)
def test_loss_counts_and_gradient(case):
    T, E, k, dtype, score, lengths, front, behind = case
    print(case, flush=True)
    z, ids = draw(T, E, k, dtype, 10 * E + T)
    off = None if lengths is None else offsets(lengths, front)
    assert off is None or off[-1] + behind == T
    loss, counts, tokens, ws = forward(z, ids, E, k, score, off)
    zf, span = z.float().cpu().numpy(), np.array([0, T]) if off is None else off
    ol, oc, on = B.balance_loss(zf, ids, score, span)
    assert np.array_equal(host(counts), oc) and np.array_equal(host(tokens), on)
    assert (np.abs(host(loss) - ol) <= (W + 4 * 1024 * U) * ol).all()
    assert m.moe_debug_check(ws) == 0
    rng = np.random.default_rng(T)
    dl = rng.standard_normal(len(span) - 1).astype(np.float32)
    oz, mag = B.balance_loss_backward(zf, oc, on, dl, k, score, span)
    half = 2.0 ** -8 if dtype == "bf16" else U
    lim = (4 * W + 64 * U) * mag
    lim = lim + half * (np.abs(oz) + lim) + 1e-36
    dz = backward(z, counts, tokens, dev_f32(dl), E, k, score, off).float().cpu().numpy()
    assert (np.abs(dz - oz)[span[0]:span[-1]] <= lim[span[0]:span[-1]]).all()
    assert (dz[:span[0]] == 9).all() and (dz[span[-1]:] == 9).all()
    into = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(z.dtype).cuda()
    before = into.float().cpu().numpy().astype(np.float64)
    dz = backward(z, counts, tokens, dev_f32(dl), E, k, score, off, acc=1, into=into).float().cpu().numpy()
    want = before + oz
    assert (np.abs(dz - want) <= (4 * W + 64 * U) * mag + (half + 2 * U) * (np.abs(before) + np.abs(oz) + lim) + 1e-36).all()
    assert (dz[:span[0]] == before[:span[0]]).all() and (dz[span[-1]:] == before[span[-1]:]).all()


@pytest.mark.parametrize("score", [B.SOFTMAX, B.SIGMOID])
def test_gradient_against_differences_of_the_device_loss(score):
    """(loss(z + h) - loss(z - h)) / 2h along the gradient itself: its norm squared, up to the loss's rounding and h^2."""
    T, E, k = 60, 12, 3
    rng = np.random.default_rng(2)
    z = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    ids = rng.integers(0, E // 2, (T, k)).astype(np.int32)
    off = offsets([25, 35], 0)
    loss, counts, tokens, _ = forward(z, ids, E, k, score, off)
    dz = backward(z, counts, tokens, torch.ones(2, device="cuda"), E, k, score, off)
    norm2, h = float(dz.double().square().sum()), 0.25
    step = dz * (h / norm2 ** 0.5)
    d = sum(float(forward(z + s * step, ids, E, k, score, off)[0].double().sum()) * s for s in (1, -1)) / (2 * h)
    # the loss: (W + 4096 u) of 2 or so, over 2 h; third derivatives: the shares' are at most 1 along a unit step, c E / (k n^2) at most 12 / 25
    assert abs(d - norm2 ** 0.5) <= 2 * (W + 4096 * U) * 3 / (2 * h) + h * h / 6 * 2


def test_strided_rows_and_untouched_neighbours():
    T, E, k, ld = 37, 40, 4, 56
    wide, ids = draw(T, E, k, "f32", 5, width=ld)
    z = wide[:, 8:8 + E]
    loss, counts, tokens, _ = forward(z, ids, E, k, B.SIGMOID, None, ldl=ld)
    dense = z.contiguous()
    l2, c2, n2, _ = forward(dense, ids, E, k, B.SIGMOID, None)
    assert torch.equal(loss, l2) and torch.equal(counts, c2) and torch.equal(tokens, n2)
    out = torch.full((T, ld), 3.0, device="cuda")
    one = torch.ones(1, device="cuda")
    backward(z, counts, tokens, one, E, k, B.SIGMOID, None, into=out[:, 8:8 + E], ldl=ld, ldd=ld)
    assert (out[:, :8] == 3).all() and (out[:, 8 + E:] == 3).all()
    assert torch.equal(out[:, 8:8 + E], backward(dense, counts, tokens, one, E, k, B.SIGMOID, None))


def test_far_sigmoids():
    """Every sigmoid of a row below float32's range: the shares are their ratios, and the gradient goes on."""
    z = np.array([[-300.0, -300.5, -301.0], [-90.0, -1000.0, -np.inf], [200.0, 100.0, -100.0]], np.float32)
    ids = np.array([[0, 1], [0, 1], [0, 1]], np.int32)
    t = torch.from_numpy(z).cuda()
    loss, counts, tokens, _ = forward(t, ids, 3, 2, B.SIGMOID, None)
    ol, oc, on = B.balance_loss(z, ids, B.SIGMOID, np.array([0, 3]))
    assert np.array_equal(host(counts), oc) and (np.abs(host(loss) - ol) <= (W + 4096 * U) * ol).all()
    dz = host(backward(t, counts, tokens, torch.ones(1, device="cuda"), 3, 2, B.SIGMOID, None))
    oz, mag = B.balance_loss_backward(z, oc, on, np.ones(1), 2, B.SIGMOID, np.array([0, 3]))
    assert (np.abs(dz - oz) <= (4 * (2 * 110 + 64) * U + 64 * U) * mag + 1e-36).all()


@pytest.mark.parametrize("off", [[0, 40, 20, 64], [-5, 10, 64], [0, 10, 90], [64, 0], [2 ** 31 - 1, -2 ** 31, 5]], ids=str)
def test_bad_offsets_are_named_and_stay_inside(off):
    T, E, k = 64, 24, 2
    z, ids = draw(T, E, k, "f32", 8)
    _, counts, tokens, ws = forward(z, ids, E, k, B.SOFTMAX, np.array(off))
    assert m.moe_debug_check(ws) == m.MOE_DEVERR_SEQUENCE
    backward(z, counts, tokens, torch.ones(len(off) - 1, device="cuda"), E, k, B.SOFTMAX, np.array(off))
    torch.cuda.synchronize()


def test_no_tokens_and_no_valid_tokens():
    E, k = 16, 2
    z = torch.full((7, E), float("-inf"), device="cuda")
    ids = np.zeros((7, k), np.int32)
    for T, off in ((0, None), (7, None), (7, np.array([0, 0, 7, 7]))):
        loss, counts, tokens, _ = forward(z[:T], ids[:T], E, k, B.SOFTMAX, off)
        assert (host(loss) == 0).all() and (host(counts) == 0).all() and (host(tokens) == 0).all()
        dz = backward(z[:T], counts, tokens, torch.ones(tokens.shape[0], device="cuda"), E, k, B.SOFTMAX, off)
        assert T == 0 or (host(dz) == 0).all()


def test_the_same_bits_every_time_and_in_a_graph():
    T, E, k = 3001, 64, 4
    off = offsets([1000, 2001], 0)
    z, ids = draw(T, E, k, "f32", 9)
    first = forward(z, ids, E, k, B.SOFTMAX, off)
    ids_d, off_d, zs = dev_i32(ids), dev_i32(off), torch.empty_like(z)
    out = [torch.empty_like(t) for t in first[:3]]
    dz, dl, ws = torch.empty_like(z), torch.rand(2, device="cuda"), first[3]

    def call():
        m.moe_balance_loss(zs, m.MOE_F32, E, ids_d, T, E, k, B.SOFTMAX, off_d, 2, *out, ws)
        m.moe_balance_loss_backward(zs, m.MOE_F32, E, out[1], out[2], dl, T, E, k, B.SOFTMAX, off_d, 2, 0, dz, E)
    zs.copy_(z)
    call()
    assert all(torch.equal(a, b) for a, b in zip(out, first))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for r in range(3):
        zs.copy_(z.roll(r, 0))
        torch.cuda.synchronize()
        g.replay()
        got = [t.clone() for t in out + [dz]]
        torch.cuda.synchronize()
        call()
        assert all(torch.equal(a, b) for a, b in zip(got, out + [dz]))
