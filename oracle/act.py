"""RMS norm with the residual's addition, SwiGLU and MXFP4 activations.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Reading.  The "RTX 4080 SUPER native Windows 27B: NInfer 80 SM port" page (its
list of hardware limits) names W4A4 matrix ops; here both operands are MXFP4
(OCP Microscaling Formats v1.0).  The activations take the weights' quantizer
(``formats.quantize_mxfp4``), and the norm and SwiGLU in front of a product are
defined as real functions rounded once to fp32 and then quantized, so that
their codes have one right value.  The arithmetic here is NumPy's extended
precision (64 significant bits), rounded once.

A 32-value block that holds a NaN or an infinity has scale 255 (E8M0 NaN) and
zero codes, or d = NaN and q = 0.
"""
import numpy as np

from . import formats as fm
from . import int8
from . import mx


def bf16(v):
    """float32 values rounded to 8 significant bits, nearest even (normals)."""
    v = np.asarray(v, dtype=np.float32).astype(np.float64)
    f, e = np.frexp(v)
    return np.ldexp(np.rint(f * 256.0), e - 8).astype(np.float32)


def _marked(X):
    """X with non-finite blocks zeroed, and which blocks those were."""
    X = np.asarray(X, dtype=np.float32)
    bad = ~np.isfinite(X.reshape(X.shape[0], -1, 32)).all(axis=-1)
    return np.where(np.repeat(bad, 32, axis=1), np.float32(0), X), bad


def quantize_mxfp4(X):
    """codes [R, K] (one E2M1 code per element) and E8M0 bytes [R, K/32]."""
    X, bad = _marked(X)
    f = fm.quantize_mxfp4(X)
    q = np.asarray(f["q"]).reshape(X.shape).astype(np.uint8)
    e = np.asarray(f["e"]).reshape(X.shape[0], -1).astype(np.uint8)
    return q, np.where(bad, 255, e).astype(np.uint8)


def pack_codes(q):
    """[R, K] codes two to a byte, low nibble first."""
    q = np.asarray(q, np.uint8)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def dequantize_mxfp4(q, e):
    """float64 values of codes [R, K] and E8M0 bytes [R, K/32] (255: NaN)."""
    e = np.asarray(e, np.int64)
    s = np.where(e == 255, np.nan, np.ldexp(1.0, np.minimum(e, 254) - 127))
    return fm.e2m1_value(q) * np.repeat(s, 32, axis=1)


def quantize(fmt, X):
    """(codes, scales) of float32 rows X in an activation format."""
    if fmt == "mxfp4":
        q, e = quantize_mxfp4(X)
        return pack_codes(q), e
    X, bad = _marked(X)
    if fmt == "mxfp8":
        q, e = mx.quantize_mxfp8(X)
        return q, np.where(bad, 255, e).astype(np.uint8)
    q, d = int8.quantize_act_q8(X)
    return q, np.where(bad, np.float32(np.nan), d)


def rms_norm(x, w, eps, res=None, res_bf16=False):
    """(y, h): h = x + res as an fp32 sum (rounded to bf16 for a bf16
    residual), y = fp32(h w / sqrt(mean h^2 + eps))."""
    x = np.asarray(x, np.float32)
    h = x
    if res is not None:
        h = (x + np.asarray(res, np.float32)).astype(np.float32)
        h = bf16(h) if res_bf16 else h
    v = h.astype(np.longdouble)
    m = (v * v).sum(axis=1, keepdims=True) / x.shape[1]
    with np.errstate(invalid="ignore", divide="ignore"):
        y = v * np.asarray(w, np.float32).astype(np.longdouble) / np.sqrt(m + np.longdouble(eps))
    return y.astype(np.float32), h


def swiglu(g, u):
    """fp32( g / (1 + exp(-g)) * u ) of finite float32 inputs."""
    g = np.asarray(g, np.float32).astype(np.longdouble)
    u = np.asarray(u, np.float32).astype(np.longdouble)
    with np.errstate(under="ignore", over="ignore"):
        return (g / (1 + np.exp(-g)) * u).astype(np.float32)


def gemm_mxfp4(W, N, K, q, e):
    """y [R, N] in float64 of packed MXFP4 weights and activation codes
    [R, K] with scales, and sum |w x| per output."""
    x = dequantize_mxfp4(q, e)
    w = fm.dequantize("mxfp4", W, N, K)
    return x @ w.T, np.abs(x) @ np.abs(w).T
