"""Buffers past 4 GiB and the widest strides: the ends of large calls hold the
bits of small calls on the same data (each checked against the oracle in the
files of its operator)."""

import pytest
import torch

import moe_fp8_grouped_amd as m

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand_u8(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8, device="cuda")


def test_rows_there_and_back():
    R, C, tail = (1 << 17) + 37, 16384 + 32, 70                  # 2.2e9 elements: 4.3 GB in, 8.6 GB back in float32
    x = torch.randn(R, C, generator=gen(1), dtype=torch.bfloat16, device="cuda")
    print("rows", R, C, flush=True)

    def there_and_back(x):
        n = x.shape[0]
        q, s = torch.zeros(n, C // 2, dtype=torch.uint8, device="cuda"), torch.zeros(n, C // 32, dtype=torch.uint8, device="cuda")
        out = torch.full((n, C), 9.0, device="cuda")
        m.moe_quantize_rows_mx4(x, None, C, m.MOE_ACT_NONE, n, C, q, C // 2, s, C // 32)
        m.moe_dequantize_rows_mx4(q, C // 2, s, C // 32, n, C, m.MOE_F32, out, C)
        return q, s, out
    big, small = there_and_back(x), there_and_back(x[-tail:])
    for a, b in zip(big, small):
        assert torch.equal(a[-tail:], b)


def test_weights():
    E, K, N = 3, 32768 + 32, 32768 + 16                          # 6.4 GB of bfloat16
    w = torch.randn(E, K, N, generator=gen(2), dtype=torch.bfloat16, device="cuda")
    print("weights", E, K, N, flush=True)

    def quantize(w):
        e = w.shape[0]
        q, s = torch.zeros(e, N, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(e, N, K // 32, dtype=torch.uint8, device="cuda")
        m.moe_quantize_weights_mx4(w, e, K, N, q, s)
        return q, s
    for a, b in zip(quantize(w), quantize(w[-1:].contiguous())):
        assert torch.equal(a[-1:], b)


@pytest.mark.parametrize("fmt", [m.MOE_MX4, m.MOE_E4M3FN])
def test_product(fmt):
    """Weights of 4.9 GB, results of 4.7 GB; the last expert's rows against a call on its window alone."""
    E, K, N, each = 72, 8192, 16384 + 16, 2000
    g = gen(3)
    w, ws = rand_u8(g, 0, 256, E, N, K // 2), rand_u8(g, 120, 128, E, N, K // 32)
    M = E * each
    if fmt == m.MOE_MX4:
        x, xs, ldl, lds = rand_u8(g, 0, 256, M, K // 2), rand_u8(g, 120, 128, M, K // 32), K // 2, K // 32
    else:
        x, xs, ldl, lds = rand_u8(g, 0, 0x70, M, K), torch.rand(M, generator=g, device="cuda"), K, 0
    sizes = torch.full((E,), each, dtype=torch.int32, device="cuda")
    print("product", fmt, M, K, N, flush=True)

    def product(x, xs, w, ws, g0, El):
        n = x.shape[0]
        out = torch.full((n, N), 9.0, dtype=torch.bfloat16, device="cuda")
        work = m.workspace(m.MOE_OP_GMM_MX4, n, K, N, E)
        m.moe_gmm_mx4(x, ldl, xs, lds, fmt, 0, w, ws, sizes, E, g0, El, n, K, N, m.MOE_BF16, out, work)
        assert m.moe_debug_check(work) == 0
        return out
    big = product(x, xs, w, ws, 0, E)
    small = product(x[-each:], xs[-each:], w[-1:], ws[-1:], E - 1, 1)
    assert torch.isfinite(small).all() and torch.equal(big[-each:], small)


@pytest.mark.parametrize("fmt", [m.MOE_MX4, m.MOE_E4M3FN])
def test_product_with_the_widest_rows(fmt):
    """Rows 2^23 bytes apart, the scales' too; 140 rows in two groups: whole tiles and a part."""
    K, N, E, ld = 416, 272, 2, 1 << 23
    g, M = gen(4), 140
    w, ws = rand_u8(g, 0, 256, E, N, K // 2), rand_u8(g, 120, 128, E, N, K // 32)
    row = K // 2 if fmt == m.MOE_MX4 else K
    x = rand_u8(g, 0, 0x70, M, row)
    wide = torch.full((M, ld), 0xFF, dtype=torch.uint8, device="cuda")
    wide[:, :row] = x
    if fmt == m.MOE_MX4:
        xs = rand_u8(g, 120, 128, M, K // 32)
        wide[:, row:row + K // 32] = xs
        xw, ldw, lds = wide[:, row:row + K // 32], ld, K // 32
    else:
        xs = torch.rand(M, generator=g, device="cuda")
        xw, ldw, lds = xs, 0, 0
    sizes = torch.tensor([131, 9], dtype=torch.int32, device="cuda")
    print("widest rows", fmt, flush=True)
    outs = []
    for a, ldl, s, l in ((x, row, xs, lds), (wide[:, :row], ld, xw, ldw)):
        out = torch.full((M, N), 9.0, device="cuda")
        m.moe_gmm_mx4(a, ldl, s, l, fmt, 0, w, ws, sizes, E, 0, E, M, K, N, m.MOE_F32, out, m.workspace(m.MOE_OP_GMM_MX4, M, K, N, E))
        outs.append(out)
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)
