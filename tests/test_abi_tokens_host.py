"""Host-side refusals of the router, the 4-bit calls and the few-token layer
(paths that return before any launch; no GPU)."""

import os

import pytest

import moe_fp8_grouped_amd as m


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoefp8.so not built")
    return m.load_library()


AL = 4096        # an aligned dummy pointer: never dereferenced on these paths


def test_router(lib):
    def f(z=AL, dt=m.MOE_F32, ldl=64, T=4, E=64, k=8, score=0, bias=None, renorm=0, scale=1.0, ids=AL, w=AL):
        return lib.moe_router_topk(z, dt, ldl, T, E, k, score, bias, renorm, scale, ids, w, None)
    for bad in (dict(E=0), dict(E=1025, ldl=2000), dict(k=0), dict(k=65, E=128, ldl=128), dict(E=4, k=5), dict(ldl=63), dict(T=-1),
                dict(T=2 ** 31 + 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert f(**bad) == m.MOE_ERR_SHAPE, bad
    for bad in (dict(dt=m.MOE_E4M3FN), dict(score=2), dict(renorm=2)):
        assert f(**bad) == m.MOE_ERR_UNSUPPORTED, bad
    for bad in (dict(z=None), dict(ids=None), dict(w=None)):
        assert f(**bad) == m.MOE_ERR_NULL, bad
    assert f(T=0, z=None) == m.MOE_OK


def test_router_backward(lib):
    def f(z=AL, dt=m.MOE_F32, ldl=64, ids=AL, dw=AL, T=4, E=64, k=8, score=0, renorm=0, scale=1.0, dz=AL, ldd=64):
        return lib.moe_router_topk_backward(z, dt, ldl, ids, dw, T, E, k, score, renorm, scale, dz, ldd, None)
    assert f(ldd=63) == m.MOE_ERR_SHAPE and f(k=65) == m.MOE_ERR_SHAPE and f(dt=7) == m.MOE_ERR_UNSUPPORTED
    for bad in (dict(z=None), dict(ids=None), dict(dw=None), dict(dz=None)):
        assert f(**bad) == m.MOE_ERR_NULL, bad
    assert f(T=0, dz=None) == m.MOE_OK


def test_quantize_rows_mx4(lib):
    def f(x=AL, up=None, ldx=64, act=0, R=4, C=64, q=AL, ldq=32, s=AL, lds=2):
        return lib.moe_quantize_rows_mx4(x, up, ldx, act, R, C, q, ldq, s, lds, None)
    for bad in (dict(C=48), dict(C=0), dict(R=-1), dict(ldx=60), dict(ldx=68), dict(ldq=16), dict(ldq=40), dict(lds=1), dict(x=AL + 2),
                dict(q=AL + 8), dict(act=1, up=AL + 4)):
        assert f(**bad) == m.MOE_ERR_SHAPE, bad
    assert f(act=2) == m.MOE_ERR_UNSUPPORTED and f(up=AL) == m.MOE_ERR_UNSUPPORTED
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(act=1)):
        assert f(**bad) == m.MOE_ERR_NULL, bad
    assert f(R=0, x=None) == m.MOE_OK


def test_quantize_weights_and_dequantize_mx4(lib):
    f = lambda w=AL, E=2, K=64, N=32, q=AL, s=AL: lib.moe_quantize_weights_mx4(w, E, K, N, q, s, None)
    for bad in (dict(K=48), dict(N=24), dict(E=-1), dict(K=0), dict(N=0), dict(w=AL + 2), dict(q=AL + 4)):
        assert f(**bad) == m.MOE_ERR_SHAPE, bad
    for bad in (dict(w=None), dict(q=None), dict(s=None)):
        assert f(**bad) == m.MOE_ERR_NULL, bad
    assert f(E=0, w=None) == m.MOE_OK
    d = lambda q=AL, ldq=32, s=AL, lds=2, R=4, C=64, dt=0, out=AL, ldo=64: lib.moe_dequantize_rows_mx4(q, ldq, s, lds, R, C, dt, out, ldo, None)
    for bad in (dict(C=48), dict(ldq=24), dict(ldq=40), dict(lds=1), dict(ldo=60), dict(ldo=68), dict(out=AL + 8), dict(R=-1)):
        assert d(**bad) == m.MOE_ERR_SHAPE, bad
    assert d(dt=m.MOE_E4M3FN) == m.MOE_ERR_UNSUPPORTED
    for bad in (dict(q=None), dict(s=None), dict(out=None)):
        assert d(**bad) == m.MOE_ERR_NULL, bad
    assert d(R=0, q=None) == m.MOE_OK


def test_gmm_mx4(lib):
    def f(lhs=AL, ldl=64, ls=AL, lds=0, fmt=m.MOE_E4M3FN, mode=0, rhs=AL, rs=AL, gs=AL, E=8, g0=0, El=8, M=16, K=64, N=32, dt=0, out=AL,
          ws=AL, wsb=1 << 30):
        return lib.moe_gmm_mx4(lhs, ldl, ls, lds, fmt, mode, rhs, rs, gs, E, g0, El, M, K, N, dt, out, ws, wsb, None)
    mx = dict(fmt=m.MOE_MX4, ldl=32, lds=2)
    for bad in (dict(K=48), dict(N=24), dict(K=0), dict(M=-1), dict(M=2 ** 31), dict(E=0), dict(E=2000), dict(g0=4, El=5), dict(ldl=48),
                dict(ldl=72), dict(lds=2), dict(mx, ldl=16), dict(mx, lds=1), dict(lhs=AL + 8), dict(rhs=AL + 8), dict(out=AL + 8),
                dict(M=2 ** 31 - 2, N=1 << 14)):
        assert f(**bad) == m.MOE_ERR_SHAPE, bad
    for bad in (dict(fmt=m.MOE_BF16), dict(mode=3), dict(mode=9), dict(mx, mode=1), dict(mx, mode=2), dict(dt=5)):
        assert f(**bad) == m.MOE_ERR_UNSUPPORTED, bad
    for bad in (dict(lhs=None), dict(ls=None), dict(rhs=None), dict(rs=None), dict(gs=None), dict(out=None)):
        assert f(**bad) == m.MOE_ERR_NULL, bad
    assert f(ws=None) == m.MOE_ERR_WORKSPACE and f(wsb=16) == m.MOE_ERR_WORKSPACE
    assert f(M=0, out=None) == m.MOE_OK


def test_ffn_tokens(lib):
    def f(x=AL, ldx=256, ids=AL, tw=AL, T=4, k=2, H=256, I=128, E=8, g0=0, El=8, fmt=m.MOE_E4M3FN, w01=AL, s01=AL, kb01=1, nb01=256, wo=AL,
          so=AL, kbo=1, nbo=256, dt=0, out=AL, ws=AL, wsb=1 << 30):
        return lib.moe_ffn_tokens(x, ldx, ids, tw, T, k, H, I, E, g0, El, fmt, w01, s01, kb01, nb01, wo, so, kbo, nbo, dt, out, ws, wsb, None)
    mx = dict(fmt=m.MOE_MX4, kb01=0, nb01=0, kbo=0, nbo=0)
    for bad in (dict(T=-1), dict(k=0), dict(H=264), dict(I=136), dict(mx, H=272, ldx=272), dict(mx, I=144), dict(ldx=248), dict(ldx=260), dict(E=0),
                dict(E=2000), dict(g0=4, El=5), dict(kb01=3), dict(nb01=3), dict(kbo=0), dict(x=AL + 2), dict(w01=AL + 8), dict(wo=AL + 8),
                dict(H=1 << 21, ldx=1 << 21)):
        assert f(**bad) == m.MOE_ERR_SHAPE, bad
    for bad in (dict(fmt=m.MOE_BF16), dict(mx, kb01=1), dict(mx, nbo=256), dict(T=65), dict(T=64, k=17), dict(kb01=4), dict(nb01=4), dict(dt=6)):
        assert f(**bad) == m.MOE_ERR_UNSUPPORTED, bad
    for bad in (dict(x=None), dict(ids=None), dict(tw=None), dict(w01=None), dict(s01=None), dict(wo=None), dict(so=None), dict(out=None)):
        assert f(**bad) == m.MOE_ERR_NULL, bad
    need = m.workspace_bytes(m.MOE_OP_FFN_TOKENS, 8, 256, 128, 8)
    assert f(ws=None) == m.MOE_ERR_WORKSPACE and f(wsb=need - 1) == m.MOE_ERR_WORKSPACE
    assert f(T=0, x=None) == m.MOE_OK


def test_workspace_sizes(lib):
    assert m.workspace_bytes(m.MOE_OP_GMM_MX4, 100, 64, 32, 8) >= 256
    a, b = (m.workspace_bytes(m.MOE_OP_FFN_TOKENS, s, 512, 256, 8) for s in (8, 512))
    assert b > a >= 256 and a % 256 == 0 and b % 256 == 0
    for bad in ((1025, 512, 256), (8, -1, 256), (8, 512, (1 << 20) + 1)):
        with pytest.raises(m.MoeError):
            m.workspace_bytes(m.MOE_OP_FFN_TOKENS, *bad, 8)


def test_alignment_of_what_is_loaded_wide(lib):
    """Scales, and the results that leave in whole vectors."""
    def g(rs=AL, fmt=m.MOE_MX4):
        return lib.moe_gmm_mx4(AL, 32, AL, 2, fmt, 0, AL, rs, AL, 8, 0, 8, 16, 64, 32, 0, AL, AL, 1 << 30, None)

    def f(s01=AL, so=AL, out=AL):
        return lib.moe_ffn_tokens(AL, 256, AL, AL, 4, 2, 256, 128, 8, 0, 8, m.MOE_MX4, AL, s01, 0, 0, AL, so, 0, 0, 0, out, AL, 1 << 30, None)
    assert g(rs=AL + 4) == m.MOE_ERR_SHAPE
    for bad in (dict(s01=AL + 2), dict(so=AL + 1), dict(out=AL + 8)):
        assert f(**bad) == m.MOE_ERR_SHAPE, bad
