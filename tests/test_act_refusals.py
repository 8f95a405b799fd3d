"""Argument checks of the norm, SwiGLU and MXFP4 entry points, on the host:
every call here is refused (or is an empty no-op) before any launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from decode_moe_mul_amd import qmoe  # noqa: E402

P = ctypes.c_void_p
OK, BAD, UNSUP = 0, -1, -2
A = 256 * 1000                       # an aligned address, never dereferenced


@pytest.fixture(scope="module")
def L():
    return qmoe.lib()


def _norm(L, fmt="mxfp4", x=A, xd=0, res=A, ro=A, rd=0, w=A, eps=1e-5, R=4, K=64, out=A, sc=A):
    return getattr(L, f"qnorm_act_{fmt}")(P(x), xd, P(res), P(ro), rd, P(w), eps, R, K, P(out),
                                          P(sc), None)


@pytest.mark.parametrize("fmt", qmoe.ACT_FORMATS)
def test_norm_act(L, fmt):
    assert _norm(L, fmt, R=0) == OK
    for bad in (dict(K=48), dict(K=0), dict(K=32800), dict(R=-1), dict(x=None), dict(w=None),
                dict(out=None), dict(sc=None), dict(x=A + 8), dict(w=A + 4), dict(out=A + 2),
                dict(res=A + 8), dict(ro=A + 8), dict(res=None), dict(eps=-1.0),
                dict(eps=float("nan"))):
        assert _norm(L, fmt, **bad) == BAD, bad
    assert _norm(L, fmt, xd=7) == UNSUP and _norm(L, fmt, rd=7) == UNSUP


def test_plain_norm(L):
    args = lambda K=64, yd=0, R=4: (P(A), 0, P(A), P(A), 0, P(A), 1e-5, R, K, P(A), yd, None)
    assert L.qnorm(*args(R=0)) == OK
    assert L.qnorm(*args(K=60)) == BAD
    assert L.qnorm(*args(yd=2)) == UNSUP


@pytest.mark.parametrize("fmt", qmoe.ACT_FORMATS)
def test_swiglu_act(L, fmt):
    def call(g=A, u=A, xd=0, ld=64, R=4, K=64, q=A, s=A):
        return getattr(L, f"qswiglu_act_{fmt}")(P(g), P(u), xd, ld, R, K, P(q), P(s), None)
    assert call(R=0) == OK
    for bad in (dict(K=40), dict(ld=32), dict(ld=68), dict(R=-1), dict(g=None), dict(u=None),
                dict(q=None), dict(s=None), dict(g=A + 8), dict(u=A + 8)):
        assert call(**bad) == BAD, bad
    assert call(xd=2) == UNSUP
    assert call(R=1 << 30, K=64) == UNSUP


def test_mxfp4_activations(L):
    q = lambda x=A, xd=0, R=4, K=64, c=A, s=A: L.qquantize_act_mxfp4(P(x), xd, R, K, P(c), P(s), None)
    d = lambda c=A, s=A, R=4, K=64, y=A, yd=0: L.qdequant_act_mxfp4(P(c), P(s), R, K, P(y), yd, None)
    assert q(R=0) == OK and d(R=0) == OK
    for bad in (dict(K=48), dict(R=-1), dict(c=None), dict(s=None), dict(c=A + 8)):
        assert q(**bad) == BAD and d(**bad) == BAD, bad
    assert q(x=None) == BAD and q(x=A + 8) == BAD and d(y=None) == BAD and d(y=A + 8) == BAD
    assert q(xd=2) == UNSUP and d(yd=2) == UNSUP
    assert q(R=1 << 30) == UNSUP and d(R=1 << 30) == UNSUP


def test_product(L):
    def g(W=A, N=16, K=64, c=A, s=A, R=4, y=A, yd=0):
        return L.qgemm_mxfp4_mxfp4(P(W), N, K, P(c), P(s), R, P(y), yd, None)
    assert g(N=0) == OK and g(R=0) == OK
    for bad in (dict(K=48), dict(K=0), dict(K=65568), dict(N=-1), dict(R=-1), dict(W=None),
                dict(c=None), dict(s=None), dict(y=None), dict(W=A + 16), dict(c=A + 8),
                dict(y=A + 4)):
        assert g(**bad) == BAD, bad
    assert g(yd=2) == UNSUP
    assert g(N=(1 << 30) + 1) == UNSUP and g(R=(1 << 30) + 1) == UNSUP
    assert g(N=1 << 20, R=1 << 24) == UNSUP           # 2^32 threads with every tile


def test_the_binding_refuses_what_the_kernels_cannot_take():
    x = torch.zeros(4, 64)
    for call in (lambda: qmoe.quantize_act_mxfp4(x),                       # host tensor
                 lambda: qmoe.norm(x, torch.ones(64), 1e-5),
                 lambda: qmoe.norm_act("q8", x, torch.ones(64), 1e-5),
                 lambda: qmoe.swiglu_act("q8", x, x),
                 lambda: qmoe.swiglu_act("q8", x, x[:, :32]),              # shapes differ
                 lambda: qmoe.swiglu_act("q8", x, x.bfloat16()),           # types differ
                 lambda: qmoe.dequantize_act_mxfp4(x, x),                  # not codes
                 lambda: qmoe.dequantize_act_mxfp4(torch.tensor(1), x),
                 lambda: qmoe.norm_act("q8", x, torch.ones(64), 1e-5, res_out=x),
                 lambda: qmoe.gemm_mxfp4_mxfp4(torch.zeros(8, dtype=torch.uint8), 16, 64,
                                               torch.zeros(4, 32, dtype=torch.uint8),
                                               torch.zeros(4, 2, dtype=torch.uint8))):
        with pytest.raises(qmoe.QmoeError):
            call()
