"""Pins of the 4-bit block oracle: the format's value set, exhaustive nearest
values, the scale rule, and the grouped product against a plain matmul."""

from fractions import Fraction

import numpy as np

from oracle import mx4
from oracle.codec import bf16_decode, e4m3_decode
from workloads import to_bf16_bits


def test_value_set():
    assert list(mx4.E2M1[:8]) == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert list(mx4.E2M1[8:]) == [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
    assert np.signbit(mx4.E2M1[8])


def test_rounding_is_nearest_even_by_exact_arithmetic():
    v = np.concatenate([np.arange(-512, 513) / 64.0, np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])])
    got = mx4.e2m1_rne(v)
    grid = [Fraction(float(x)) for x in mx4.E2M1[:8]]
    for x, c in zip(v, got):
        a = abs(Fraction(float(x)))
        d = [abs(a - g) for g in grid]
        best = [i for i in range(8) if d[i] == min(d)]
        want = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
        assert c & 7 == want, (x, c)
        assert bool(c & 8) == bool(np.signbit(x))


def test_scale_brings_the_largest_into_its_binade():
    rng = np.random.default_rng(3)
    v = bf16_decode(to_bf16_bits((rng.standard_normal((200, 32)) * np.exp2(rng.integers(-100, 100, (200, 1)))).astype(np.float32)))
    q, s = mx4.quantize_values(v)
    top = np.abs(v.astype(np.float64)).max(-1) / np.ldexp(1.0, s[:, 0].astype(np.int64) - 127)
    assert ((top >= 4) & (top < 8)).all()
    back = mx4.decode(q, s)
    # nearest value: half a step of the block's binade, or the saturation of (6, 8)
    err = np.abs(back - v) / np.ldexp(1.0, s.astype(np.int64) - 127)
    assert err.max() < 2.0
    inside = np.abs(v) / np.ldexp(1.0, s.astype(np.int64) - 127) <= 6
    assert err[inside].max() <= 1.0


def test_special_blocks():
    v = np.zeros((5, 32))
    v[0, :] = -0.0
    v[1, 3] = np.inf
    v[2, 4] = np.nan
    v[3, 0] = 2.0 ** -133
    v[4, 0] = 2.0 ** 127
    q, s = mx4.quantize_values(v)
    assert s[:, 0].tolist() == [127, 255, 255, 0, 252]
    assert (mx4.unpack(q[0]) == 8).all()
    assert np.isnan(mx4.decode(q[1:3], s[1:3])).all()
    assert mx4.decode(q[4:], s[4:])[0, 0] == 2.0 ** 127


def test_pack_round_trip():
    codes = np.random.default_rng(0).integers(0, 16, (7, 64)).astype(np.uint8)
    assert (mx4.unpack(mx4.pack(codes)) == codes).all()
    assert mx4.pack(codes)[0, 0] == codes[0, 0] + 16 * codes[0, 1]


def test_gmm_against_a_matmul_of_the_values():
    rng = np.random.default_rng(5)
    K, N, gs = 96, 48, np.array([3, 0, 5, 2])
    x = rng.integers(0, 0x7f, (10, K)).astype(np.uint8)
    ls = rng.random(10).astype(np.float32)
    w = rng.standard_normal((4, N, K))
    q, s = mx4.quantize_values(w)
    o, A = mx4.gmm_mx4(x, ls, q, s, gs, 0, 4)
    W = mx4.decode(q, s)
    owner = np.repeat(np.arange(4), gs)
    want = np.stack([ls[r].astype(np.float64) * (W[owner[r]] @ e4m3_decode(x[r])) for r in range(10)])
    assert np.allclose(o, want, rtol=1e-12, atol=1e-12) and (A >= np.abs(o) - 1e-9).all()
    o2, _ = mx4.gmm_mx4(x[:7], ls[:7], q[1:3], s[1:3], gs, 1, 2, M=9)
    want2 = np.stack([ls[r].astype(np.float64) * (W[2] @ e4m3_decode(x[r])) for r in range(5)])
    assert np.allclose(o2[:5], want2) and (o2[5:] == 0).all()
