"""Host-side refusals of the b128 calls and of the balance loss (paths that
return before any launch; no GPU)."""

import os

import pytest

import moe_fp8_grouped_amd as m


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libmoefp8.so not built")
    return m.load_library()


AL = 4096        # an aligned dummy pointer: never dereferenced on these paths
BIG = 1 << 62


def check(f, shape=(), unsupported=(), null=(), workspace=(), ok=()):
    for bad in shape:
        assert f(**bad) == m.MOE_ERR_SHAPE, bad
    for bad in unsupported:
        assert f(**bad) == m.MOE_ERR_UNSUPPORTED, bad
    for bad in null:
        assert f(**bad) == m.MOE_ERR_NULL, bad
    for bad in workspace:
        assert f(**bad) == m.MOE_ERR_WORKSPACE, bad
    for good in ok:
        assert f(**good) == m.MOE_OK, good


def test_quantize_rows(lib):
    def f(x=AL, up=None, ldx=144, act=0, R=4, C=144, q=AL, ldq=160, s=AL, lds=2):
        return lib.moe_quantize_rows_b128(x, up, ldx, act, R, C, q, ldq, s, lds, None)
    check(f, [dict(C=136), dict(C=0), dict(C=1 << 32, ldx=1 << 33, ldq=1 << 33, lds=1 << 30), dict(R=-1), dict(ldx=136), dict(ldx=148),
              dict(ldq=128), dict(ldq=152), dict(lds=1), dict(x=AL + 2), dict(q=AL + 8), dict(act=1, up=AL + 4)],
          [dict(act=2), dict(up=AL)], [dict(x=None), dict(q=None), dict(s=None), dict(act=1)], ok=[dict(R=0, x=None)])


def test_quantize_weights(lib):
    def f(w=AL, E=2, K=64, N=32, q=AL, s=AL, qt=AL, st=AL):
        return lib.moe_quantize_weights_b128(w, E, K, N, q, s, qt, st, None)
    check(f, [dict(K=40), dict(N=24), dict(E=-1), dict(K=0), dict(N=0), dict(N=1 << 40), dict(w=AL + 2), dict(q=AL + 4), dict(qt=AL + 4)],
          null=[dict(w=None), dict(q=None), dict(s=None), dict(qt=None), dict(st=None), dict(q=None, s=None, qt=None, st=None)],
          ok=[dict(E=0, w=None)])


def test_quantize_cols(lib):
    def f(x=AL, up=None, ldx=64, act=0, T=8, k=2, perm=AL, gs=AL, E=8, g0=0, El=8, M=16, C=64, qt=AL, st=AL, ws=AL, wsb=256):
        return lib.moe_quantize_cols_b128(x, up, ldx, act, T, k, perm, gs, E, g0, El, M, C, qt, st, ws, wsb, None)
    check(f, [dict(C=40), dict(C=0), dict(C=BIG), dict(M=-1), dict(M=1 << 23), dict(M=(1 << 23) - 8), dict(M=BIG), dict(ldx=48), dict(ldx=68), dict(T=-1),
              dict(T=1 << 31), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(g0=-1), dict(g0=4, El=5), dict(El=-1),
              dict(perm=None, T=15), dict(x=AL + 8), dict(qt=AL + 8), dict(st=AL + 8), dict(act=1, up=AL + 8)],
          [dict(act=3), dict(up=AL)], [dict(x=None), dict(gs=None), dict(qt=None), dict(st=None), dict(act=1)],
          [dict(ws=None), dict(wsb=255)], [dict(M=0, x=None), dict(El=0, x=None), dict(T=0, x=None)])


def test_gmm(lib):
    def f(lhs=AL, ldl=144, ls=AL, lds=16, rhs=AL, rs=AL, sdt=m.MOE_E8M0, gs=AL, E=8, g0=0, El=8, M=16, K=144, N=32, dt=0, out=AL, ws=AL,
          wsb=1 << 40):
        return lib.moe_gmm_b128(lhs, ldl, ls, lds, rhs, rs, sdt, gs, E, g0, El, M, K, N, dt, out, ws, wsb, None)
    check(f, [dict(K=136), dict(N=24), dict(K=0), dict(N=0), dict(M=-1), dict(M=2 ** 31), dict(M=BIG), dict(K=(1 << 22) + 16, ldl=1 << 23, lds=1 << 16),
              dict(N=BIG), dict(E=0), dict(E=2000), dict(g0=4, El=5), dict(ldl=128), dict(ldl=152), dict(ldl=(1 << 23) + 16), dict(ldl=(1 << 22) + 16), dict(lds=0), dict(lds=8),
              dict(K=2064, ldl=2064), dict(lds=(1 << 23) + 16), dict(lhs=AL + 8), dict(ls=AL + 8), dict(rhs=AL + 8), dict(out=AL + 8),
              dict(sdt=m.MOE_F32, rs=AL + 2), dict(M=2 ** 31 - 2, N=1 << 14)],
          [dict(sdt=m.MOE_BF16), dict(sdt=9), dict(dt=5)],
          [dict(lhs=None), dict(ls=None), dict(rhs=None), dict(rs=None), dict(gs=None), dict(out=None)],
          [dict(ws=None), dict(wsb=0)], [dict(M=0, lhs=None, out=None)])


def test_tgmm(lib):
    def f(x=AL, xs=AL, y=AL, ys=AL, gs=AL, E=8, g0=0, El=8, M=16, K=144, N=32, dt=0, out=AL, ws=AL, wsb=1 << 40):
        return lib.moe_tgmm_b128(x, xs, y, ys, gs, E, g0, El, M, K, N, dt, out, ws, wsb, None)
    check(f, [dict(K=136), dict(N=24), dict(K=0), dict(N=0), dict(K=BIG), dict(N=BIG), dict(M=-1), dict(M=1 << 23), dict(M=BIG), dict(E=0), dict(E=2000),
              dict(g0=4, El=5), dict(x=AL + 8), dict(xs=AL + 8), dict(y=AL + 8), dict(ys=AL + 8), dict(out=AL + 8), dict(K=1 << 20, N=1 << 20)],
          [dict(dt=5), dict(dt=m.MOE_E4M3FN)], [dict(x=None), dict(xs=None), dict(y=None), dict(ys=None), dict(gs=None), dict(out=None)],
          [dict(ws=None), dict(wsb=0)], [dict(El=0, x=None, out=None)])


def test_balance_loss(lib):
    def f(z=AL, dt=m.MOE_F32, ldl=64, ids=AL, T=4, E=64, k=8, score=0, off=AL, S=2, loss=AL, c=AL, n=AL, ws=AL, wsb=1 << 40):
        return lib.moe_balance_loss(z, dt, ldl, ids, T, E, k, score, off, S, loss, c, n, ws, wsb, None)
    check(f, [dict(E=0), dict(E=1025, ldl=2000), dict(k=0), dict(k=65, E=128, ldl=128), dict(E=4, k=5), dict(ldl=63), dict(T=-1), dict(T=2 ** 31),
              dict(T=BIG), dict(S=0), dict(S=(1 << 24) + 1)],
          [dict(dt=m.MOE_E4M3FN), dict(score=2)],
          [dict(z=None), dict(ids=None), dict(loss=None), dict(c=None), dict(n=None), dict(off=None)],
          [dict(ws=None), dict(wsb=m.workspace_bytes(m.MOE_OP_BALANCE, 4, 2, 0, 64) - 1)])


def test_balance_loss_backward(lib):
    def f(z=AL, dt=m.MOE_F32, ldl=64, c=AL, n=AL, dl=AL, T=4, E=64, k=8, score=0, off=AL, S=2, acc=0, dz=AL, ldd=64):
        return lib.moe_balance_loss_backward(z, dt, ldl, c, n, dl, T, E, k, score, off, S, acc, dz, ldd, None)
    check(f, [dict(ldd=63), dict(k=65), dict(ldl=63), dict(S=0), dict(T=2 ** 31)], [dict(dt=7), dict(score=2), dict(acc=2)],
          [dict(z=None), dict(c=None), dict(n=None), dict(dl=None), dict(dz=None), dict(off=None)], ok=[dict(T=0, dz=None)])


def test_workspaces(lib):
    for op in (m.MOE_OP_GMM_B128, m.MOE_OP_TGMM_B128):
        b = m.workspace_bytes(op, 4096, 2048, 1536, 64)
        assert b >= 256 and b % 256 == 0
        with pytest.raises(m.MoeError):
            m.workspace_bytes(op, -1, 64, 64, 8)
    small, large = m.workspace_bytes(m.MOE_OP_BALANCE, 0, 1, 0, 8), m.workspace_bytes(m.MOE_OP_BALANCE, 8192, 4, 0, 256)
    assert 256 <= small < large and small % 256 == large % 256 == 0
    for bad in ((-1, 1, 8), (2 ** 31, 1, 8), (8, 0, 8), (8, 1, 0), (8, 1, 1025)):
        with pytest.raises(m.MoeError):
            m.workspace_bytes(m.MOE_OP_BALANCE, bad[0], bad[1], 0, bad[2])


P, WS = AL, 1 << 30
WINDOWS = {      # every call here that takes a window of groups, with no rows
    "moe_quantize_cols_b128": lambda f, w: f(P, None, 64, 0, 0, 2, P, P, *w, 0, 64, P, P, P, WS, None),
    "moe_gmm_b128": lambda f, w: f(P, 64, P, 16, P, P, m.MOE_E8M0, P, *w, 0, 64, 32, 0, P, P, WS, None),
    "moe_tgmm_b128": lambda f, w: f(P, P, P, P, P, *w, 0, 64, 32, 0, P, P, WS, None),
}


@pytest.mark.parametrize("name", WINDOWS)
def test_windows(lib, name):
    f = getattr(lib, name)
    big = 2 ** 31 - 1
    for w in ((8, 4, 5), (8, -1, 2), (8, 2, -1), (8, 9, 0), (8, big, 1), (8, big - 7, 8), (8, 8, big), (1024, big - 1023, 1024), (1, big, big),
              (0, 0, 0), (1025, 0, 1)):
        assert WINDOWS[name](f, w) == m.MOE_ERR_SHAPE, w


def test_every_call_of_blocks_with_a_window_is_listed():
    with open(m.HEADER_PATH) as f:
        decls = [d.split("*/")[-1] for d in f.read().split(";")]
    assert {d.split("(")[0].split()[-1] for d in decls if "int32_t first_group" in d} == set(WINDOWS)
