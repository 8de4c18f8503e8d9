"""Pins of the b128 oracle: against exact rational arithmetic, nearest-value
search, torch's float8 cast and brute force (no GPU)."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import b128
from oracle.codec import bf16_decode, e4m3_decode
from workloads import to_bf16_bits

E4M3 = np.array([e4m3_decode(np.uint8(c)) for c in range(127)], np.float64)      # finite magnitudes, ascending


def test_scale_is_the_smallest_power_of_two_that_holds_the_block():
    bits = np.arange(0x7F80, dtype=np.uint32)                                    # every finite bf16 magnitude
    amax = bf16_decode(bits.astype(np.uint16)).astype(np.float64)
    code = b128.scale_codes(amax).astype(np.int64)
    assert code[0] == 127 and code.max() <= 247
    for a, c in list(zip(amax, code))[1::7]:
        a = Fraction(float(a))
        assert a <= 448 * Fraction(2) ** int(c - 127)
        assert c == 0 or a > 448 * Fraction(2) ** int(c - 128)


def test_a_block_that_is_not_finite_is_nan_with_codes_zero():
    v = np.ones((3, 256))
    v[0, 5], v[1, 130], v[2, 0] = np.inf, np.nan, -np.inf
    q, s = b128.quantize_values(v)
    assert s.tolist() == [[255, 119], [119, 255], [255, 119]]
    assert (q[0, :128] == 0).all() and (q[1, 128:] == 0).all() and (q[0, 128:] != 0).all()
    assert np.isnan(b128.scale_values(s)).sum() == 3


@pytest.mark.parametrize("R,C", [(1, 16), (3, 128), (4, 144), (2, 400)])
def test_rows_against_nearest_value_search_and_torch(R, C):
    rng = np.random.default_rng(R * C)
    xb = to_bf16_bits((rng.standard_normal((R, C)) * 10.0 ** rng.uniform(-30, 30, (R, 1))).astype(np.float32))
    q, s = b128.quantize_rows_b128(xb)
    x = bf16_decode(xb).astype(np.float64)
    for r in range(R):
        for b in range(-(-C // 128)):
            v = x[r, 128 * b:128 * b + 128]
            p = Fraction(2) ** int(int(s[r, b]) - 127)
            assert max(Fraction(float(abs(t))) for t in v) <= 448 * p
            for t, code in zip(v, q[r, 128 * b:128 * b + 128]):
                y = float(Fraction(float(t)) / p)
                d = np.abs(E4M3 - abs(y))
                near = np.flatnonzero(d == d.min())
                want = near[0] if near.size == 1 else near[near % 2 == 0][0]
                assert (int(code) & 127) == want and (int(code) >> 7) == int(np.signbit(t))
            y = torch.from_numpy((v / float(p)).astype(np.float32)).to(torch.float8_e4m3fn)
            assert np.array_equal(y.view(torch.uint8).numpy(), q[r, 128 * b:128 * b + 128])


def test_weights_are_rows_of_their_blocks_in_both_orientations():
    rng = np.random.default_rng(3)
    wb = to_bf16_bits((rng.standard_normal((2, 144, 272)) * 0.02).astype(np.float32))
    q, s = b128.quantize_weights_b128(wb)
    qt, st = b128.quantize_weights_b128(np.ascontiguousarray(wb.transpose(0, 2, 1)))
    assert np.array_equal(q.transpose(0, 2, 1), qt) and np.array_equal(s.transpose(0, 2, 1), st)
    w = bf16_decode(wb).astype(np.float64)
    for e, a, b in ((0, 0, 0), (1, 1, 2), (0, 1, 1)):
        t = w[e, 128 * a:128 * a + 128, 128 * b:128 * b + 128]
        q1, s1 = b128.quantize_values(np.concatenate([t.reshape(-1)[:128]] * 1).reshape(1, -1))
        assert s1[0, 0] <= s[e, a, b] and s[e, a, b] == b128.scale_codes(np.abs(t).max())


def test_columns_are_rows_of_the_transpose_by_group():
    rng = np.random.default_rng(5)
    gs = np.array([4, 0, 130, 1, 128, 60, -3, 2])
    v = rng.standard_normal((200, 48))
    cols = 256 * -(-(200 + 128 * 8) // 256)
    qt, st, written = b128.quantize_cols_b128(v, gs, 1, 5, 200, cols)     # groups of 0, 130, 1, 128 -> 69 rows, 60 -> 0
    assert written.sum() == 128 * (2 + 1 + 1)
    r = p = 0
    for m in (0, 130, 1, 69, 0):
        if m:
            q, s = b128.quantize_values(np.ascontiguousarray(v[r:r + m].T))
            n = 128 * s.shape[1]
            assert np.array_equal(qt[:, p:p + m], q) and (qt[:, p + m:p + n] == 0).all()
            assert np.array_equal(st[p // 128:(p + n) // 128].T, s)
            p += n
        r += m


def test_products_against_brute_force():
    rng = np.random.default_rng(9)
    gs, M, K, N = np.array([3, 0, 5, 2]), 9, 160, 144
    x = rng.integers(0, 127, (M, K)).astype(np.uint8) | (rng.integers(0, 2, (M, K)).astype(np.uint8) << 7)
    w = rng.integers(0, 127, (3, N, K)).astype(np.uint8)
    xs, ws = rng.integers(120, 134, (M, 2)).astype(np.uint8), rng.integers(120, 134, (3, 2, 2)).astype(np.uint8)
    out, A = b128.gmm_b128(x, xs, w, ws, gs, 1, 3, M)
    group = [1] * 5 + [2] * 2                                # local groups of 0, 5, 2 rows
    for r in range(M):
        for n in (0, 5, 127, 128, 143):
            t = [Fraction(float(e4m3_decode(x[r, k]))) * Fraction(2) ** (int(xs[r, k // 128]) - 127) *
                 Fraction(float(e4m3_decode(w[group[r], n, k]))) * Fraction(2) ** (int(ws[group[r], k // 128, n // 128]) - 127)
                 for k in range(K)] if r < 7 else [Fraction(0)]
            assert abs(out[r, n] - float(sum(t))) <= 1e-12 * float(sum(abs(v) for v in t))
            assert abs(A[r, n] - float(sum(abs(v) for v in t))) <= 1e-12 * A[r, n]
    f = (rng.random((3, 2, 2)) + 0.5).astype(np.float32)
    out, _ = b128.gmm_b128(x, np.full((M, 2), 127, np.uint8), w, f, gs, 1, 3, M)
    want = sum(float(e4m3_decode(x[6, k])) * float(e4m3_decode(w[2, 130, k])) * float(f[2, k // 128, 1]) for k in range(K))
    assert np.isclose(out[6, 130], want, rtol=1e-12)


def test_weight_gradient_against_brute_force():
    rng = np.random.default_rng(11)
    gs, M, K, N = np.array([3, 0, 150]), 153, 16, 32
    cols = 256 * -(-(M + 128 * 3) // 256)
    x, y = rng.standard_normal((M, K)), rng.standard_normal((M, N))
    (xq, xs, _), (yq, ys, _) = (b128.quantize_cols_b128(v, gs, 0, 3, M, cols) for v in (x, y))
    out, A = b128.tgmm_b128(xq, xs, yq, ys, gs, 0, 3, M)
    assert (out[1] == 0).all()
    for g, r0, m, p0 in ((0, 0, 3, 0), (2, 3, 150, 128)):
        for k, n in ((0, 0), (15, 31), (7, 3)):
            want = sum(float(e4m3_decode(xq[k, p0 + i])) * float(b128.scale_values(xs[(p0 + i) // 128, k])) *
                       float(e4m3_decode(yq[n, p0 + i])) * float(b128.scale_values(ys[(p0 + i) // 128, n])) for i in range(m))
            assert abs(out[g, k, n] - want) <= 1e-12 * A[g, k, n]
    # and near the unquantized one: two roundings of half a step, 2^-4 each, per term
    dense = np.stack([x[:3].T @ y[:3], np.zeros((K, N)), x[3:].T @ y[3:]])
    mag = np.stack([np.abs(x[:3].T) @ np.abs(y[:3]), np.zeros((K, N)), np.abs(x[3:].T) @ np.abs(y[3:])])
    small = 2.0 ** -9                                         # elements below the format's normal range: half its least step, times a scale below 2^-6
    assert (np.abs(out - dense) <= (2 * 2.0 ** -4 + 2.0 ** -8) * mag + small * 153).all()
