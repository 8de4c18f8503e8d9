"""Which kernel a product in blocks of 128 runs: the cases of the GPU tests are
asked of the library's own rule, so that a change of its limits cannot move
one to another kernel unseen."""

import pytest

from tests import b128_rule as rule
from tests import test_gpu_b128_kernels as K

pytestmark = pytest.mark.skipif(rule.compiler() is None, reason="no host compiler")


@pytest.mark.parametrize("case", K.PRODUCT + K.ONE_GROUP + [K.NARROW_FAR], ids=K.ident)
def test_products_run_the_kernel_they_name(case):
    kernel, gs, g0, El, _, N, spare = case
    assert rule.product_kernel(El, sum(gs[g0:g0 + El]) + spare, N) == kernel


@pytest.mark.parametrize("case", K.GRADIENT, ids=K.ident)
def test_gradients_run_the_kernel_they_name(case):
    kernel, gs, _, El, Kdim, N = case
    assert rule.gradient_kernel(El, Kdim, N) == kernel


def test_every_kernel_is_named():
    assert {c[0] for c in K.PRODUCT} == set(rule.KERNELS) and {c[0] for c in K.GRADIENT} == {"narrow", "wide"}


def test_a_case_has_more_tiles_a_workgroup_than_it_decodes_at_a_time():
    _, gs, _, _, _, N, _ = K.PRODUCT[-1]
    assert sum(-(-n // 320) for n in gs) * -(-N // 256) > 64 * rule.CUS


def test_the_rule_at_its_borders():
    # six pieces of 16 by 16 a CU
    assert rule.product_kernel(1, 16, 16 * 1536) == "few16" and rule.product_kernel(1, 16, 16 * 1537) != "few16"
    assert rule.product_kernel(1, 17, 16 * 768) == "few32" and rule.product_kernel(1, 17, 16 * 769) == "narrow"
    assert rule.product_kernel(1, 33, 16 * 384) == "few64" and rule.product_kernel(1, 33, 16 * 385) == "narrow"
    # a wide tile for every workgroup
    assert rule.product_kernel(64, 16320, 256 * 2) == "narrow" and rule.product_kernel(128, 40960, 256) == "wide"
    assert rule.gradient_kernel(255, 256, 256) == "narrow" and rule.gradient_kernel(256, 16, 16) == "wide"
    # no local expert, and more experts than rows
    assert rule.product_kernel(0, 5, 32) == "few16" and rule.product_kernel(1000, 3, 1024) == "few16"


@pytest.mark.parametrize("cus", [8, 15, 32, 80, 228, 256, 304])
def test_narrow_tiles_are_decoded_at_once(cus):
    """However the rows fall, a workgroup of the narrow kernel has at most the 64 tiles that its table holds: the worst split of M
    rows into El groups makes M / 64 + groups row tiles, and an XCD's share of all tiles goes to cus / 8 workgroups at least."""
    import random
    rng, worst = random.Random(cus), 0
    for _ in range(20000):
        El, M, N = rng.choice((1, 2, 3, 8, 32, 64, 256, 1000)), int(2 ** rng.uniform(0, 17)), 16 * int(2 ** rng.uniform(0, 10))
        if rule.product_kernel(El, M, N, cus) == "narrow":
            worst = max(worst, -(-((M // 64 + min(El, M)) * -(-N // 64)) // 8) / (cus // 8))
        Kdim = 16 * int(2 ** rng.uniform(0, 10))
        if rule.gradient_kernel(El, Kdim, N, cus) == "narrow":
            worst = max(worst, -(-(El * -(-Kdim // 64) * -(-N // 64)) // 8) / (cus // 8))
    assert 2 < worst and -(-worst // 1) <= 64


def test_the_large_layer_runs_the_wide_kernels():
    from tests.test_gpu_block_scaled_ffn_wide import CASE
    M, El, H, I = CASE["T"] * CASE["k"], CASE["El"], CASE["H"], CASE["I"]
    products = [2 * I, H, I, H]                             # forward up and down, then to h and to x
    kernels = [rule.product_kernel(El, M, N) for N in products] + [rule.gradient_kernel(El, I, H), rule.gradient_kernel(El, H, 2 * I)]
    assert kernels == ["wide", "wide", "narrow", "wide", "wide", "wide"], kernels
