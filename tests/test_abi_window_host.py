"""Host-side refusal of a window of local experts that is not one: its end is
formed without passing 32 bits (paths that return before any launch; no GPU)."""

import os

import pytest

import moe_fp8_grouped_amd as m

P = 4096         # an aligned dummy pointer: never dereferenced on these paths
WS = 1 << 30

# every entry point that takes a window, with no tokens and no rows
CALLS = {
    "moe_sort_by_expert": lambda f, w: f(P, 0, 2, *w, P, P, 0, 64, 0, P, P, P, P, P, P, WS, None),
    "moe_sort_by_expert_noalloc": lambda f, w: f(P, 0, 2, *w, P, P, 0, 64, 0, P, P, P, P, P, P, None),
    "moe_quantize_sort_by_expert": lambda f, w: f(P, 0, 64, 0, 0.0, P, 2, *w, 0, P, P, P, P, P, None, None, P, WS, None),
    "moe_gmm_fp8": lambda f, w: f(P, P, 0, P, P, 1, 128, 0, P, *w, 0, 128, 128, 0, P, P, WS, None),
    "moe_gmm_i8": lambda f, w: f(P, P, 0, P, P, 1, 128, 0, P, *w, 0, 128, 128, 0, P, P, WS, None),
    "moe_tgmm_fp8": lambda f, w: f(P, P, 1, P, P, 1, P, *w, 0, 128, 128, 0, P, P, WS, None),
    "moe_tgmm_fp8_xt": lambda f, w: f(P, P, 1, P, P, 1, P, *w, 0, 256, 128, 0, P, P, WS, None),
    "moe_sort_gather_transposed": lambda f, w: f(P, 0, 0.0, 0, 2, 256, P, P, *w, 0, P, P, P, WS, None),
    "moe_gather_reduce_backward": lambda f, w: f(P, P, P, P, 0, 2, 64, P, *w, 0, P, P, None, None, None, None),
    "moe_gmm_mx4": lambda f, w: f(P, 64, P, 0, m.MOE_E4M3FN, 0, P, P, P, *w, 0, 64, 32, 0, P, P, WS, None),
    "moe_ffn_tokens": lambda f, w: f(P, 256, P, P, 0, 2, 256, 128, *w, m.MOE_MX4, P, P, 0, 0, P, P, 0, 0, 0, P, P, WS, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_windows(name):
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoefp8.so not built")
    f = getattr(m.load_library(), name)
    big = 2 ** 31 - 1
    for w in ((8, 4, 5), (8, -1, 2), (8, 2, -1), (8, 9, 0), (8, big, 1), (8, big - 7, 8), (8, 8, big), (1024, big - 1023, 1024), (1, big, big),
              (0, 0, 0), (1025, 0, 1)):
        assert CALLS[name](f, w) == m.MOE_ERR_SHAPE, w


def test_every_call_with_a_window_is_listed():
    with open(m.HEADER_PATH) as f:
        decls = [d.split("*/")[-1] for d in f.read().split(";")]
    takes = {d.split("(")[0].split()[-1] for d in decls if "int32_t group_offset" in d}
    assert takes == set(CALLS)
