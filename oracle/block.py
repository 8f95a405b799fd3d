"""The dense block's fused products and norms.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Products in float64 of what the codes stand for, every output with the sum of
|w x| that bounds its rounding errors, activation functions with their slopes, and
the norms around a block in NumPy's extended precision (64 significant bits),
rounded where the definition rounds.
"""
import math

import numpy as np

from . import act as a4
from . import formats as fm
from . import int8
from . import mx

WEIGHTS = {"q8": "q8_0", "mxfp8": "mxfp4", "mxfp4": "mxfp4"}
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def values(fmt, codes, scales):
    """float64 values of activations as the library lays them out."""
    if fmt == "q8":
        return int8.dequantize_act_q8(codes, scales)
    if fmt == "mxfp8":
        return mx.dequantize_mxfp8(codes, scales)
    codes = np.asarray(codes, np.uint8)
    q = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[0], -1)
    return a4.dequantize_mxfp4(q, scales)


def product(fmt, W, N, K, codes, scales):
    """(x W^T, |x| |W|^T) in float64."""
    x, w = values(fmt, codes, scales), fm.dequantize(WEIGHTS[fmt], W, N, K)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def activation(name, v):
    """(f(v), a bound on |f'| near v) in float64."""
    v = np.asarray(v, np.float64)
    one = np.ones_like(v)
    if name in (None, "none"):
        return v, one
    if name == "relu":
        return np.maximum(v, 0), one
    if name == "relu2":
        return np.maximum(v, 0) ** 2, 2 * np.abs(v) + 1e-3
    with np.errstate(over="ignore", under="ignore"):
        if name == "silu":
            return v / (1 + np.exp(-v)), 1.1 * one
        if name == "gelu":
            return 0.5 * v * _erfc(-v * math.sqrt(0.5)), 1.13 * one
        u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        return v / (1 + np.exp(-2 * u)), 1.13 * one


def stream(x, res, w_post=None, eps_post=0.0, gate=None, scale=1.0, res_scale=1.0):
    """res_scale res + scale gate z before its rounding, z = x w_post / sqrt(mean x^2 +
    eps_post) or x, and the sum of its two terms' magnitudes."""
    L = np.longdouble
    z = np.asarray(x, np.float32).astype(L)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        if w_post is not None:
            m = (z * z).sum(axis=1, keepdims=True) / z.shape[1]
            z = z * np.asarray(w_post, np.float32).astype(L) / np.sqrt(m + L(eps_post))
        if gate is not None:
            g = np.asarray(gate, np.float32).reshape(-1, z.shape[1]).astype(L)
            z = z * np.repeat(g, z.shape[0] // g.shape[0], axis=0)
        a, b = L(res_scale) * np.asarray(res, np.float32).astype(L), L(scale) * z
        return a + b, np.abs(a) + np.abs(b)


def rounded(h, bf):
    """h in float32, and from there in bfloat16."""
    with np.errstate(over="ignore", invalid="ignore"):
        h = np.asarray(h).astype(np.float32)
        return a4.bf16(h) if bf else h


def norm_block(x, res, w, eps, w_post=None, eps_post=0.0, gate=None, scale=1.0, res_scale=1.0,
               res_bf16=False):
    """(y, h): h is the stream rounded to float32 (and to bf16), y = fp32(h w /
    sqrt(mean h^2 + eps))."""
    h = rounded(stream(x, res, w_post, eps_post, gate, scale, res_scale)[0], res_bf16)
    return a4.rms_norm(h, w, eps)[0], h
