"""The oracle of the dense block's products and norms against its definitions."""
import math

import numpy as np
import pytest

from oracle import act
from oracle import block
from oracle import formats as fm
from oracle import int8
from oracle import mx

ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


@pytest.mark.parametrize("fmt", ("q8", "mxfp8", "mxfp4"))
def test_product_is_the_sum_over_k(fmt):
    rng = np.random.default_rng(1)
    R, N, K = 3, 5, 64
    x = rng.normal(size=(R, K)).astype(np.float32)
    w = rng.normal(size=(N, K)).astype(np.float32)
    W = fm.quantize(block.WEIGHTS[fmt], w)
    codes, scales = act.quantize(fmt, x)
    y, bound = block.product(fmt, W, N, K, codes, scales)
    v = block.values(fmt, codes, scales)
    want = {"q8": lambda: int8.dequantize_act_q8(*int8.quantize_act_q8(x)),
            "mxfp8": lambda: mx.dequantize_mxfp8(*mx.quantize_mxfp8(x)),
            "mxfp4": lambda: act.dequantize_mxfp4(*act.quantize_mxfp4(x))}[fmt]()
    assert (v == want).all()
    deq = fm.dequantize(block.WEIGHTS[fmt], W, N, K)
    for r in range(R):
        for n in range(N):
            terms = [v[r, k] * deq[n, k] for k in range(K)]
            assert math.isclose(y[r, n], math.fsum(terms), rel_tol=0, abs_tol=1e-12)
            assert math.isclose(bound[r, n], math.fsum(map(abs, terms)), rel_tol=1e-12)


def test_activations_at_known_points():
    f = lambda name, v: float(block.activation(name, np.array([v]))[0][0])
    assert f("none", -3.0) == -3.0 and f("relu", -3.0) == 0.0 and f("relu", 2.0) == 2.0
    assert f("relu2", 3.0) == 9.0 and f("relu2", -3.0) == 0.0
    assert math.isclose(f("silu", 1.0), 1 / (1 + math.exp(-1)))
    assert math.isclose(f("gelu", 1.0), 0.5 * (1 + math.erf(math.sqrt(0.5))))
    u = math.sqrt(2 / math.pi) * 1.044715
    assert math.isclose(f("gelu_tanh", 1.0), 0.5 * (1 + math.tanh(u)))
    assert math.isclose(f("gelu_tanh", -2.0),
                        -(1 + math.tanh(-math.sqrt(2 / math.pi) * (2 + 0.044715 * 8))))


@pytest.mark.parametrize("name", ACTS)
def test_slopes_bound_the_differences(name):
    v = np.linspace(-9, 9, 4001)
    f, slope = block.activation(name, v)
    assert (np.abs(np.diff(f)) <= np.maximum(slope[1:], slope[:-1]) * np.diff(v) + 1e-12).all()


def test_norm_block_without_post_norm_gate_and_scales_is_the_norm():
    rng = np.random.default_rng(2)
    x, res = (rng.normal(size=(4, 96)).astype(np.float32) for _ in range(2))
    w = rng.normal(size=96).astype(np.float32)
    for bf in (False, True):
        a = block.norm_block(x, res, w, 1e-5, res_bf16=bf)
        b = act.rms_norm(x, w, 1e-5, res, res_bf16=bf)
        assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


def test_norm_block_by_hand():
    rng = np.random.default_rng(3)
    R, K, G = 6, 32, 3
    x, res = (rng.normal(size=(R, K)).astype(np.float32) for _ in range(2))
    w, wp = (rng.normal(size=K).astype(np.float32) for _ in range(2))
    gate = rng.normal(size=(G, K)).astype(np.float32)
    y, h = block.norm_block(x, res, w, 1e-3, wp, 1e-2, gate, 0.5, 1.5)
    for r in range(R):
        m = math.fsum(float(v) ** 2 for v in x[r]) / K
        hs = [1.5 * float(res[r, k]) + 0.5 * float(gate[r // (R // G), k]) * float(x[r, k])
              * float(wp[k]) / math.sqrt(m + 1e-2) for k in range(K)]
        assert np.allclose(h[r], hs, rtol=1e-7, atol=1e-7)
        m = math.fsum(float(v) ** 2 for v in h[r]) / K
        ys = [float(h[r, k]) * float(w[k]) / math.sqrt(m + 1e-3) for k in range(K)]
        assert np.allclose(y[r], ys, rtol=1e-7, atol=1e-7)
