"""Pins of the norm, SwiGLU and MXFP4-activation references: closed forms,
scalar loops and the format's definition."""
import math

import numpy as np
import pytest

from oracle import act
from oracle import formats as fm


def test_mxfp4_closed_forms():
    x = np.zeros((3, 64), np.float32)
    x[0, :8] = [4.0, 2.5, -2.5, 3.5, 0.25, 0.75, -0.25, 5.0]   # E = 0
    x[1, 0] = 7.9                                              # above 6: saturates
    x[1, 32:] = 1.0                                            # E = -2: 4 = code 6
    q, e = act.quantize_mxfp4(x)
    # 2.5 -> 2 (code 4), 3.5 -> 4 (6), 0.25 -> 0, 0.75 -> 1 (2), 5 -> 4: ties to even codes
    assert q[0, :8].tolist() == [6, 4, 8 + 4, 6, 0, 2, 8, 6]
    assert e.tolist() == [[127, 0], [127, 125], [0, 0]]
    assert q[1, 0] == 7 and (q[1, 32:] == 6).all() and (q[2] == 0).all()
    assert act.dequantize_mxfp4(q, e)[0, :8].tolist() == [4, 2, -2, 4, 0, 1, 0, 4]
    assert act.pack_codes(q)[0, :2].tolist() == [6 | 4 << 4, 12 | 6 << 4]


def test_a_negative_value_that_vanishes_in_its_block_keeps_its_sign():
    x = np.zeros((1, 32), np.float32)
    x[0, :3] = [1e30, -1e-30, -0.0]
    assert act.quantize("mxfp4", x)[0][0, :2].tolist() == [0x87, 0x00]
    assert act.quantize("mxfp8", x)[0][0, :3].tolist() == [125, 128, 0]


@pytest.mark.parametrize("fmt", ["q8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("v", [np.nan, np.inf, -np.inf])
def test_a_non_finite_block_is_marked_alone(fmt, v):
    x = np.ones((1, 96), np.float32)
    x[0, 40] = v
    q, s = act.quantize(fmt, x)
    clean, cs = act.quantize(fmt, np.ones((1, 96), np.float32))
    w = q.shape[1] // 3
    assert (q[0, w:2 * w] == 0).all()
    assert np.isnan(s[0, 1]) if fmt == "q8" else s[0, 1] == 255
    assert (q[0, :w] == clean[0, :w]).all() and (q[0, 2 * w:] == clean[0, 2 * w:]).all()
    assert s[0, 0] == cs[0, 0] and s[0, 2] == cs[0, 2]


def test_bf16_rounds_to_nearest_even():
    v = np.array([1.0, 1 + 2 ** -8, 1 + 3 * 2 ** -8, 1 + 2 ** -8 + 2 ** -20, -3.0, 0.0], np.float32)
    assert act.bf16(v).tolist() == [1.0, 1.0, 1 + 2 ** -6, 1 + 2 ** -7, -3.0, 0.0]


def test_rms_norm_against_a_scalar_loop():
    rng = np.random.default_rng(1)
    x, r = rng.normal(0, 1, (2, 3, 40)).astype(np.float32)
    w = rng.normal(1, 0.1, 40).astype(np.float32)
    y, h = act.rms_norm(x, w, 1e-5, r)
    for i in range(3):
        hs = [float(np.float32(a + b)) for a, b in zip(x[i], r[i])]
        m = math.fsum(v * v for v in hs) / 40
        for j in range(40):
            assert h[i, j] == np.float32(hs[j])
            assert y[i, j] == pytest.approx(hs[j] * float(w[j]) / math.sqrt(m + 1e-5), rel=2 ** -23)
    assert act.rms_norm(np.zeros((1, 32)), np.ones(32), 1e-6)[0].tolist() == [[0.0] * 32]


def test_swiglu_against_scalars():
    g = np.array([[-1000.0, -3.0, 0.0, 0.5, 20.0, 1000.0]], np.float32)
    u = np.array([[2.0, 1.5, 7.0, -2.0, 1.0, 3.0]], np.float32)
    got = act.swiglu(g, u)[0]
    assert got[0] == 0.0 and got[2] == 0.0 and got[5] == 3000.0
    for i in (1, 3, 4):
        want = g[0, i] / (1 + math.exp(-float(g[0, i]))) * u[0, i]
        assert got[i] == pytest.approx(want, rel=2 ** -23)


def test_product_against_scalars():
    rng = np.random.default_rng(2)
    N, K, R = 3, 64, 2
    buf = fm.quantize("mxfp4", rng.normal(0, 1, (N, K)).astype(np.float32))
    q, e = act.quantize_mxfp4(rng.normal(0, 1, (R, K)))
    y, bound = act.gemm_mxfp4(buf, N, K, q, e)
    w = fm.dequantize("mxfp4", buf, N, K)
    for r in range(R):
        for n in range(N):
            terms = [float(w[n, k]) * float(fm.e2m1_value(q[r, k])) * 2.0 ** (int(e[r, k // 32]) - 127)
                     for k in range(K)]
            assert y[r, n] == pytest.approx(math.fsum(terms), abs=1e-12)
            assert bound[r, n] == pytest.approx(math.fsum(abs(t) for t in terms))


def test_int8_is_within_one_step_of_the_int8_quantizer():
    """The two differ in the last bit of d alone."""
    from oracle import int8
    x = np.random.default_rng(3).normal(0, 1, (40, 320)).astype(np.float32)
    x[0] = 0
    q, d = act.quantize("q8", x)
    q0, d0 = int8.quantize_act_q8(x)
    assert (np.abs(d - d0) <= 2 * np.spacing(d0)).all() and (q[0] == 0).all() and (d[0] == 0).all()
    assert (np.abs(q.astype(int) - q0) <= 1).all() and (q != q0).mean() < 1e-3
    assert (np.abs(q.reshape(40, 10, 32)).max(-1)[1:] == 127).all()


def test_int8_is_the_int8_quantizer():
    from oracle import int8
    x = np.random.default_rng(4).normal(0, 1, (400, 320)).astype(np.float32)
    x[0], x[1] = 0, 1e-44
    (q, d), (q0, d0) = act.quantize("q8", x), int8.quantize_act_q8(x)
    assert (q == q0).all() and (d == d0).all()
    assert (d == (np.abs(x.reshape(400, 10, 32)).max(-1) / np.float32(127))).all()
