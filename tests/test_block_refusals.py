"""Argument checks of the fused products and the norms around a block, on the host:
every call here is refused (or is an empty no-op) before any launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from decode_moe_mul_amd import qmoe  # noqa: E402

P = ctypes.c_void_p
OK, BAD, UNSUP = 0, -1, -2
A = 256 * 1000                       # an aligned address, never dereferenced
FMTS = qmoe.ACT_FORMATS


@pytest.fixture(scope="module")
def L():
    return qmoe.lib()


def test_the_entry_points_are_exported(L):
    for f in FMTS:
        for name in (f"qlinear_{f}", f"qglu_{f}", f"qglu_{f}_act", f"qnorm_block_act_{f}"):
            assert hasattr(L, name)
    assert hasattr(L, "qnorm_block")


@pytest.mark.parametrize("fmt", FMTS)
def test_linear(L, fmt):
    def f(W=A, N=16, K=64, c=A, s=A, R=4, b=A, act=1, r=A, rd=0, y=A + 4096, yd=0):
        return getattr(L, f"qlinear_{fmt}")(P(W), N, K, P(c), P(s), R, P(b), act, P(r), rd, P(y),
                                            yd, None)
    assert f(N=0) == OK and f(R=0) == OK
    for bad in (dict(K=48), dict(K=0), dict(K=65568), dict(N=-1), dict(R=-1), dict(W=None),
                dict(c=None), dict(s=None), dict(y=None), dict(W=A + 16), dict(c=A + 8),
                dict(y=A + 4), dict(b=A + 2), dict(r=A + 8), dict(r=A, y=A, rd=1, yd=0)):
        assert f(**bad) == BAD, bad
    assert f(yd=2) == UNSUP and f(yd=1 << 20) == UNSUP and f(rd=7) == UNSUP
    assert f(act=-1) == UNSUP and f(act=6) == UNSUP
    assert f(N=(1 << 30) + 1) == UNSUP and f(R=(1 << 30) + 1) == UNSUP
    assert f(N=1 << 20, R=1 << 24) == UNSUP           # 2^32 threads with every tile
    if fmt == "q8":
        assert f(s=A + 2) == BAD


@pytest.mark.parametrize("fmt", FMTS)
def test_glu(L, fmt):
    def f(W=A, U=A, N=32, K=64, c=A, s=A, R=4, b=A, b2=A, act=1, y=A, yd=0):
        return getattr(L, f"qglu_{fmt}")(P(W), P(U), N, K, P(c), P(s), R, P(b), P(b2), act, P(y),
                                         yd, None)

    def g(W=A, U=A, N=32, K=64, c=A, s=A, R=4, b=A, b2=A, act=1, y=A, ys=A):
        return getattr(L, f"qglu_{fmt}_act")(P(W), P(U), N, K, P(c), P(s), R, P(b), P(b2), act,
                                             P(y), P(ys), None)
    for call in (f, g):
        assert call(N=0) == OK and call(R=0) == OK
        for bad in (dict(K=48), dict(K=0), dict(K=65568), dict(N=-1), dict(R=-1), dict(W=None),
                    dict(U=None), dict(c=None), dict(s=None), dict(y=None), dict(W=A + 16),
                    dict(U=A + 128), dict(c=A + 8), dict(y=A + 4), dict(b=A + 2), dict(b2=A + 1)):
            assert call(**bad) == BAD, bad
        assert call(act=-1) == UNSUP and call(act=6) == UNSUP
        assert call(N=(1 << 30) + 32) == UNSUP and call(R=(1 << 30) + 1) == UNSUP
    assert f(yd=2) == UNSUP and f(yd=1 << 20) == UNSUP and f(yd=-1) == UNSUP
    assert g(N=48) == BAD and g(ys=None) == BAD
    if fmt == "q8":
        assert g(ys=A + 2) == BAD


def _nb(L, name, out, x=A, xd=0, wp=A, ep=1e-5, g=A, gd=0, G=2, sc=1.0, r=A, ro=A, rd=0, rs=1.0,
        w=A, eps=1e-5, R=4, K=64):
    return getattr(L, name)(P(x), xd, P(wp), ep, P(g), gd, G, sc, P(r), P(ro), rd, rs, P(w), eps,
                            R, K, *out, None)


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_block_act(L, fmt):
    f = lambda q=A, s=A, **kw: _nb(L, f"qnorm_block_act_{fmt}", (P(q), P(s)), **kw)
    assert f(R=0) == OK
    for bad in (dict(K=48), dict(K=0), dict(K=32800), dict(R=-1), dict(x=None), dict(w=None),
                dict(r=None), dict(q=None), dict(s=None), dict(x=A + 8), dict(w=A + 4),
                dict(wp=A + 4), dict(g=A + 8), dict(r=A + 8), dict(ro=A + 8), dict(q=A + 2),
                dict(eps=-1.0), dict(eps=float("nan")), dict(ep=-1.0), dict(G=3), dict(G=0),
                dict(G=-2), dict(G=8)):
        assert f(**bad) == BAD, bad
    for bad in (dict(xd=7), dict(rd=7), dict(gd=7)):
        assert f(**bad) == UNSUP, bad
    if fmt == "q8":
        assert f(s=A + 2) == BAD


def test_plain_norm_block(L):
    f = lambda yd=0, **kw: _nb(L, "qnorm_block", (P(A), yd), **kw)
    assert f(R=0) == OK
    assert f(K=60) == BAD
    assert f(yd=2) == UNSUP


def test_the_binding_refuses_what_the_kernels_cannot_take():
    x = torch.zeros(4, 64)
    w = torch.ones(64)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    W = torch.zeros(4096, dtype=torch.uint8)
    for call in (lambda: qmoe.linear("mxfp4", W, 16, 64, c, s),              # host tensors
                 lambda: qmoe.linear("fp8", W, 16, 64, c, s),
                 lambda: qmoe.linear("mxfp4", W, 16, 64, c, s, act="swish"),
                 lambda: qmoe.linear("mxfp4", W, 16, 60, c, s),
                 lambda: qmoe.linear("mxfp4", W, -1, 64, c, s),
                 lambda: qmoe.glu("mxfp8", W, W, 16, 64, c, s),              # codes of another format
                 lambda: qmoe.glu("q8", W, W, 16, 64, c, s),
                 lambda: qmoe.glu_act("mxfp4", W, W, 16, 64, c, s),
                 lambda: qmoe.norm_block(x, x, w, 1e-5),
                 lambda: qmoe.norm_block_act("q8", x, x, w, 1e-5)):
        with pytest.raises(qmoe.QmoeError):
            call()
