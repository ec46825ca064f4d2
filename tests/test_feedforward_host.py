"""The feed-forward operators' checks that need no GPU: every refusal returns before the library touches one, and the
addresses are never read."""
import ctypes as C

import pytest

EINVAL, ESHAPE, EALIGN, EUNSUPPORTED, EWORKSPACE = 1, 2, 3, 4, 9
A, B, D, F, H = (C.c_void_p(n << 32) for n in range(1, 6))   # far from one another
ODD = C.c_void_p((9 << 32) + 1)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    return g.lib()


def test_norm(L):
    def norm(x=A, dtype=0, T=2, K=64, xs=64, rest=None, rs=64, total=None, ts=64, w=B, wt=0, eps=1e-6, y=D, yt=0, ys=64,
             q=None, d=None):
        return L.rfp2_rms_norm(x, dtype, T, K, xs, rest, rs, total, ts, w, wt, eps, y, yt, ys, q, d, None)

    assert norm(T=0, x=None) == 0 and norm(K=0) == 0
    assert [norm(x=None), norm(w=None), norm(y=None), norm(dtype=3), norm(wt=-1), norm(yt=5), norm(T=-1), norm(q=F), norm(d=F),
            norm(eps=0.0), norm(eps=-1.0), norm(eps=NAN), norm(eps=INF), norm(total=F)] == [EINVAL] * 14
    assert [norm(K=32769), norm(K=40, q=F, d=H), norm(T=1 << 32), norm(ys=63), norm(rest=F, total=H, ts=3), norm(xs=-64)] == [ESHAPE] * 6
    assert [norm(x=ODD), norm(w=ODD), norm(y=ODD, yt=1), norm(rest=ODD), norm(q=ODD, d=F), norm(q=F, d=ODD)] == [EALIGN] * 6
    # outputs over inputs and over one another, but for whole rows in their own place
    next_row = C.c_void_p((1 << 32) + 256)
    assert [norm(y=next_row), norm(y=A, yt=1), norm(y=A, ys=128), norm(y=B), norm(rest=F, total=H, y=H), norm(rest=F, total=B),
            norm(q=A, d=F), norm(q=F, d=F), norm(q=F, d=D)] == [EINVAL] * 9


def test_route(L):
    def route(x=A, dtype=0, T=2, E=64, stride=64, scoring=0, bias=None, groups=1, keep=1, top=1, k=4, scale=1.0, ids=B, w=D):
        return L.rfp2_moe_route(x, dtype, T, E, stride, scoring, bias, groups, keep, top, k, 1, scale, ids, w, None)

    assert route(T=0, x=None) == 0
    assert [route(x=None), route(ids=None), route(w=None), route(dtype=9), route(scoring=2), route(scoring=-1), route(T=-1),
            route(scale=NAN), route(scale=INF)] == [EINVAL] * 9
    assert [route(E=0), route(E=1025), route(k=0), route(k=33), route(E=3), route(groups=0), route(groups=3), route(groups=64, keep=4),
            route(groups=4, keep=5), route(groups=4, keep=0), route(top=0), route(top=3), route(T=1 << 32), route(stride=-1)] == [ESHAPE] * 14
    assert [route(x=ODD), route(bias=ODD), route(ids=ODD), route(w=ODD)] == [EALIGN] * 4
    assert [route(ids=A), route(w=A), route(ids=B, w=B), route(bias=B), route(bias=D)] == [EINVAL] * 5


def test_combine(L):
    def combine(y=A, dtype=0, T=2, k=2, M=64, yt=128, yj=64, w=B, ids=None, rest=None, rs=64, out=D, ot=0, os=64):
        return L.rfp2_moe_combine(y, dtype, T, k, M, yt, yj, w, ids, rest, rs, out, ot, os, None)

    assert combine(T=0, y=None) == 0 and combine(M=0) == 0
    assert [combine(y=None), combine(w=None), combine(out=None), combine(dtype=4), combine(ot=-1), combine(T=-1), combine(M=-1)] == [EINVAL] * 7
    assert [combine(k=0), combine(k=1025), combine(T=1 << 32), combine(M=1 << 32), combine(os=63), combine(rest=F, rs=-1),
            combine(yt=-1), combine(yj=-64)] == [ESHAPE] * 8
    assert [combine(y=ODD), combine(w=ODD), combine(ids=ODD), combine(rest=ODD), combine(out=ODD)] == [EALIGN] * 5
    assert [combine(out=B), combine(ids=D), combine(rest=C.c_void_p((3 << 32) + 256)), combine(rest=D, rs=128), combine(out=A),
            combine(out=C.c_void_p((1 << 32) + 256 * 3))] == [EINVAL] * 6


def test_moe_gemm(L):
    def gemm(W=A, E=4, M=64, K=256, ids=B, T=2, k=2, X=D, bias=None, act=0, Y=F, ws=H, n=1 << 20):
        return L.rfp2_moe_gemm(W, E, M, K, ids, T, k, X, 0, bias, act, Y, ws, n, None, None)

    assert gemm(T=0, W=None) == 0
    assert [gemm(W=None), gemm(ids=None), gemm(X=None), gemm(Y=None), gemm(T=-1), gemm(act=3), gemm(act=-1)] == [EINVAL] * 7
    assert [gemm(E=0), gemm(E=1025), gemm(M=0), gemm(K=0), gemm(k=0), gemm(T=1 << 24), gemm(E=1024, M=1 << 21), gemm(K=1 << 21)] == [ESHAPE] * 8
    assert [gemm(K=128), gemm(M=24), gemm(M=48, act=1)] == [EUNSUPPORTED] * 3
    assert [gemm(ws=None), gemm(n=16)] == [EWORKSPACE] * 2
    assert [gemm(W=ODD), gemm(ids=ODD), gemm(X=ODD), gemm(bias=ODD), gemm(Y=ODD), gemm(ws=C.c_void_p((9 << 32) + 16))] == [EALIGN] * 6
    assert [gemm(Y=A), gemm(Y=B), gemm(Y=D), gemm(ws=F), gemm(ws=B), gemm(Y=C.c_void_p((5 << 32) + 256))] == [EINVAL] * 6


def test_workspace_sizes():
    import gemm_rocmfp2_mul_gb300 as g
    assert g.rfp2_moe_gemm_workspace_bytes(0, 8, 16) == 0
    small, large = g.rfp2_moe_gemm_workspace_bytes(16, 8, 256), g.rfp2_moe_gemm_workspace_bytes(16384, 8, 256)
    assert 0 < small < large < 1 << 21
