"""The dense block's fused products (bias, activation, residual, gated pairs) and
the norms around a block, against the 64-bit oracle, alone and run together."""
import numpy as np
import pytest

from gpu_util import requires_gpu, to_gpu, to_np, assert_bitexact, torch
from oracle import act
from oracle import block
from oracle import formats as fm
from decode_moe_mul_amd import qmoe, synth

pytestmark = [pytest.mark.gpu, requires_gpu]
FMTS = qmoe.ACT_FORMATS
ACTS = (None, "silu", "gelu", "gelu_tanh", "relu", "relu2")
EPS = 2.0 ** -24


def _normal(shape, seed, sigma=1.0, bf=False):
    x = synth.normal(shape, sigma, seed, synth.ACT, shape[0])
    return synth.bf16_round(x) if bf else x


def _dev(x, bf=False):
    return None if x is None else to_gpu(x).to(torch.bfloat16) if bf else to_gpu(x)


def _dtype(bf):
    return torch.bfloat16 if bf else torch.float32


# ------------------------------------------------------------- operands --

def _grid_weights(rng, fmt, N, K):
    """Packed weights of few binary places: sums of their products with
    _grid_activations are exact in fp32 in any order."""
    nb = K // 32
    if fmt == "q8":
        return fm.pack("q8_0", {"q": rng.integers(-12, 13, (N, nb, 32)).astype(np.int8),
                                "d": (2.0 ** rng.integers(-1, 2, (N, nb))).astype(np.float16)},
                       N, K)
    return fm.pack("mxfp4", {"q": rng.integers(0, 16, (N, K)).astype(np.uint8),
                             "e": rng.integers(126, 129, (N, nb)).astype(np.uint8)}, N, K)


def _grid_activations(rng, fmt, R, K):
    if fmt == "q8":
        return (rng.integers(-12, 13, (R, K)).astype(np.int8),
                (2.0 ** rng.integers(-1, 2, (R, K // 32))).astype(np.float32))
    e = rng.integers(126, 129, (R, K // 32)).astype(np.uint8)
    if fmt == "mxfp4":
        return act.pack_codes(rng.integers(0, 16, (R, K)).astype(np.uint8)), e
    # 0 .. 15 in halves, of either sign: eight products span fewer than 13 binary places
    codes = np.array([0, 0x30, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4A, 0x4C, 0x50, 0x52, 0x57],
                     np.uint8)
    return (codes[rng.integers(0, len(codes), (R, K))]
            | (rng.integers(0, 2, (R, K)) << 7).astype(np.uint8)), e


def _real(fmt, R, N, K, seed, pair=False):
    """Quantized normal activations and weights on the GPU and on the host."""
    x = _normal((R, K), seed) * np.exp2(
        np.random.default_rng(seed).integers(-3, 2, (R, 1))).astype(np.float32)
    codes, scales = act.quantize(fmt, x)
    W = [fm.quantize(block.WEIGHTS[fmt], synth.normal((N, K), 1.0 / np.sqrt(K), seed, synth.GATE, i))
         for i in range(2 if pair else 1)]
    return W, codes, scales


def _sums(fmt, W, N, K, codes, scales, f32):
    """Exact sums and how far the kernel's may be: fp32 sums of exact terms in any
    order; of MXFP8 with a result not in fp32, seven of eight products lose less
    than 2^-13 of the largest each."""
    y, b = block.product(fmt, W, N, K, codes, scales)
    rel = K * EPS + (0 if f32 or fmt != "mxfp8" else 2.0 ** -10)
    return y, rel * b


def _activated(name, v, e):
    """The activation of sums v known to within e, and its own error."""
    f, _ = block.activation(name, v)
    # the slope's bound holds around v; relu2's grows with it
    slope = block.activation(name, np.abs(v) + e)[1]
    own = 0 if name in (None, "relu") else (2.0 ** -20) * (1 + v * v / 4) * np.abs(f) + 2.0 ** -118
    return f, slope * e + own


def _close(got, want, err, bf, what=""):
    """|got - want| <= err and the rounding of the result to its type."""
    half = np.abs(want) * 2.0 ** (-8 if bf else -24) + (2.0 ** -134 if bf else 2.0 ** -150)
    lim = err * (1 + 2.0 ** -7) + half
    d = np.abs(to_np(got.float()).astype(np.float64) - want)
    assert got.shape == want.shape and (d <= lim).all(), \
        f"{what}: {(~(d <= lim)).sum()} of {d.size} off, worst {np.nanmax(d / lim):.3g} of the bound"


# rows around every kernel's tile, widths that end inside one, K of one block, K that
# ends inside a step and inside a turn
SHAPES = [(1, 32, 32), (1, 1, 64), (1, 2050, 4096), (2, 49, 6752), (6, 640, 2048), (15, 130, 416),
          (16, 256, 512), (17, 33, 1056), (33, 640, 2048), (64, 2048, 640), (65, 100, 544),
          (130, 258, 1120), (257, 384, 224), (300, 515, 2080), (513, 1030, 160), (5, 9001, 288),
          (300, 2001, 1312), (700, 2600, 352), (1000, 3900, 544), (2000, 4003, 800),
          (2040, 8100, 256), (2047, 8101, 288)]
SMALL = [(1, 40, 96), (6, 132, 544), (16, 70, 1056), (40, 100, 288), (130, 258, 1120),
         (300, 66, 160), (1100, 1030, 96)]


# ------------------------------------------------------------- products --

@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_linear_on_an_exact_grid(R, N, K, fmt, bf):
    """Terms are multiples of 2^-4 (q8 2^-2) and sums of their magnitudes below 2^20
    (2^22), so that every order of summation gives the oracle's value to the bit; a
    wrong pairing of values, blocks, scales, rows or columns changes it."""
    rng = np.random.default_rng(R * 7 + N + K)
    W, (c, s) = _grid_weights(rng, fmt, N, K), _grid_activations(rng, fmt, R, K)
    bias = rng.integers(-8, 9, N).astype(np.float32)
    res = rng.integers(-64, 65, (R, N)).astype(np.float32)
    y, b = block.product(fmt, W, N, K, c, s)
    assert b.max() < 2.0 ** (22 if fmt == "q8" else 20) - 128
    gw, gc, gs = to_gpu(W), to_gpu(c), to_gpu(s)
    out = lambda v: act.bf16(v.astype(np.float32)) if bf else v
    got = qmoe.linear(fmt, gw, N, K, gc, gs, dtype=_dtype(bf))
    assert_bitexact(to_np(got.float()), out(y), "plain")
    got = qmoe.linear(fmt, gw, N, K, gc, gs, bias=to_gpu(bias), act="relu",
                      res=_dev(res, not bf), dtype=_dtype(bf))
    assert_bitexact(to_np(got.float()), out(np.maximum(y + bias, 0) + res), "epilogue")


@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_glu_on_an_exact_grid(R, N, K, fmt, bf):
    rng = np.random.default_rng(R * 5 + N + K)
    W = [_grid_weights(rng, fmt, N, K) for _ in range(2)]
    c, s = _grid_activations(rng, fmt, R, K)
    bias = rng.integers(-8, 9, (2, N)).astype(np.float32)
    g, u = (block.product(fmt, w, N, K, c, s)[0] for w in W)
    args = (fmt, to_gpu(W[0]), to_gpu(W[1]), N, K, to_gpu(c), to_gpu(s))
    out = lambda v: act.bf16(v.astype(np.float32)) if bf else v.astype(np.float32)
    got = qmoe.glu(*args, act=None, dtype=_dtype(bf))
    assert_bitexact(to_np(got.float()), out(g * u), "plain")
    got = qmoe.glu(*args, act="relu", bias_gate=to_gpu(bias[0]), bias_up=to_gpu(bias[1]),
                   dtype=_dtype(bf))
    assert_bitexact(to_np(got.float()), out(np.maximum(g + bias[0], 0) * (u + bias[1])), "biases")


_SEPARATE = {"q8": qmoe.quantize_act_q8, "mxfp8": qmoe.quantize_act_mxfp8,
             "mxfp4": qmoe.quantize_act_mxfp4}


@pytest.mark.parametrize("R,N,K", [(r, -(-n // 32) * 32, k) for r, n, k in SHAPES])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", [None, "silu"])
def test_glu_quantized_is_the_quantizer_on_glu(R, N, K, fmt, name):
    """On exact sums the fp32 rows are the same, whatever kernel computes them, and
    so are their codes and scales."""
    rng = np.random.default_rng(R * 3 + N + K)
    W = [to_gpu(_grid_weights(rng, fmt, N, K)) for _ in range(2)]
    c, s = (to_gpu(t) for t in _grid_activations(rng, fmt, R, K))
    want = _SEPARATE[fmt](qmoe.glu(fmt, *W, N, K, c, s, act=name))
    got = qmoe.glu_act(fmt, *W, N, K, c, s, act=name)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])


@pytest.mark.parametrize("R,N,K", SMALL)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_linear_random(R, N, K, fmt, name, bf):
    (W,), c, s = _real(fmt, R, N, K, 3)
    bias, res = _normal((1, N), 4, 0.5)[0], _normal((R, N), 5, 3.0, bf=bf)
    v, e = _sums(fmt, W, N, K, c, s, not bf)
    gw, gc, gs = to_gpu(W), to_gpu(c), to_gpu(s)
    f, fe = _activated(name, v, e)
    got = qmoe.linear(fmt, gw, N, K, gc, gs, act=name, dtype=_dtype(bf))
    _close(got, f, fe, bf, "no bias, no residual")
    f, fe = _activated(name, v + bias, e + EPS * (np.abs(v) + np.abs(bias)))
    fe = fe + EPS * (np.abs(f) + fe + np.abs(res))
    got = qmoe.linear(fmt, gw, N, K, gc, gs, bias=to_gpu(bias), act=name, res=_dev(res, bf),
                      dtype=_dtype(bf))
    _close(got, f + res, fe, bf, "bias and residual")


@pytest.mark.parametrize("R,N,K", SMALL)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_glu_random(R, N, K, fmt, name, bf):
    W, c, s = _real(fmt, R, N, K, 6, pair=True)
    bias = _normal((2, N), 7, 0.5)
    (g, ge), (u, ue) = (_sums(fmt, w, N, K, c, s, not bf) for w in W)
    for b, gb, ub in ((0, None, None), (1, bias[0], bias[1])):
        gv, uv = (g, u) if not b else (g + gb, u + ub)
        add = lambda v, w, e: e + b * EPS * (np.abs(v) + np.abs(bias[w]))
        f, fe = _activated(name, gv, add(g, 0, ge))
        e2 = add(u, 1, ue)
        err = fe * (np.abs(uv) + e2) + np.abs(f) * e2
        err = err + EPS * (np.abs(f * uv) + err)
        got = qmoe.glu(fmt, to_gpu(W[0]), to_gpu(W[1]), N, K, to_gpu(c), to_gpu(s), act=name,
                       bias_gate=_dev(gb), bias_up=_dev(ub), dtype=_dtype(bf))
        _close(got, f * uv, err, bf, f"biases {b}")


@pytest.mark.parametrize("R", [3, 40, 300])
def test_mxfp8_of_every_size_in_one_block(R):
    """fp32 results keep the smallest codes beside the largest: 448 and 2^-9 in turn,
    where the matrix op alone would drop the small ones' products."""
    N, K = 96, 256
    rng = np.random.default_rng(2)
    c = rng.integers(0, 0x7F, (R, K)).astype(np.uint8)      # every finite magnitude
    c[:, ::2], c[:, 1::8] = 0x7E, 1
    c |= (rng.integers(0, 2, (R, K)) << 7).astype(np.uint8)
    s = np.full((R, K // 32), 127, np.uint8)
    W = _grid_weights(rng, "mxfp4", N, K)
    y, b = block.product("mxfp8", W, N, K, c, s)
    got = qmoe.linear("mxfp8", to_gpu(W), N, K, to_gpu(c), to_gpu(s))
    _close(got, y, K * EPS * b, False)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("R", [2, 40])
def test_activations_over_their_whole_range(R, name):
    """Sums chosen one by one: a weight row of one product each, and activations
    of 0 and 1, so that the bias is what the function sees."""
    K, v = 32, np.concatenate([np.linspace(-12, 12, 2401), np.linspace(-200, 200, 401),
                               [-1e30, 1e30, -3e38, 3e15, -1e-30, 1e-40, 0.0]]).astype(np.float32)
    if name == "relu2":
        v = np.clip(v, -3e38, 1e15).astype(np.float32)
    N = v.size
    W, c = np.zeros(fm.tensor_bytes("mxfp4", N, K), np.uint8), np.zeros((R, K // 2), np.uint8)
    s = np.full((R, 1), 127, np.uint8)
    got = qmoe.linear("mxfp4", to_gpu(W), N, K, to_gpu(c), to_gpu(s), bias=to_gpu(v), act=name)
    d = v.astype(np.float64)
    f, err = _activated(name, d, 0.0)
    with np.errstate(over="ignore", invalid="ignore"):
        _close(got, np.broadcast_to(f, (R, N)), np.broadcast_to(err, (R, N)) + 0.0, False, str(name))


@pytest.mark.parametrize("name", ACTS)
def test_infinite_and_nan_sums(name):
    v = np.array([np.inf, -np.inf, np.nan, 1.0], np.float32)
    W, c = np.zeros(fm.tensor_bytes("mxfp4", 4, 32), np.uint8), np.zeros((2, 16), np.uint8)
    y = to_np(qmoe.linear("mxfp4", to_gpu(W), 4, 32, to_gpu(c),
                          to_gpu(np.full((2, 1), 127, np.uint8)), bias=to_gpu(v), act=name))
    assert (y[:, 0] == np.inf).all() and np.isnan(y[:, 2]).all() and np.isfinite(y[:, 3]).all()
    low = {None: -np.inf, "relu": 0.0, "relu2": 0.0}
    assert (y[:, 1] == low[name]).all() if name in low else np.isnan(y[:, 1]).all()


# few rows in one and in several groups, then every int8 tile
@pytest.mark.parametrize("R,N", [(2, 140), (16, 140), (40, 140), (100, 4160), (300, 2008),
                                 (700, 2600), (1000, 3900), (2000, 4003)])
def test_int8_scales_at_the_ends_of_their_types(R, N):
    """A weight scale that is infinite makes its row's results infinite, as the formula
    does, and no other; a marked block makes its row NaN; scales of fp16's and fp32's
    subnormals count."""
    K, nb = 160, 5
    q, qx = np.ones((N, nb, 32), np.int8), np.ones((R, K), np.int8)
    d = np.ones((N, nb), np.float16)
    d[3, 2], d[130, 4] = np.inf, -np.inf
    d[64] = 2.0 ** -24
    dx = np.ones((R, nb), np.float32)
    dx[R - 1] = 2.0 ** -120
    dx[0, nb - 1] = np.nan
    W = to_gpu(fm.pack("q8_0", {"q": q, "d": d}, N, K))
    want = 32.0 * (dx.astype(np.float64) @ d.T.astype(np.float64))  # exact in fp32
    assert np.isnan(want[0]).all() and not np.isnan(want[1:]).any()
    y = qmoe.linear("q8", W, N, K, to_gpu(qx), to_gpu(dx))
    assert np.array_equal(to_np(y), want.astype(np.float32), equal_nan=True)
    y = qmoe.glu("q8", W, W, N, K, to_gpu(qx), to_gpu(dx), act=None, bias_up=to_gpu(
        np.full(N, 1.0, np.float32)))
    f = want.astype(np.float32)
    one = f + np.float32(1)  # integers and tiny values: one rounding
    assert np.array_equal(to_np(y), f * one, equal_nan=True)


# ------------------------------------------ rows, marks, aliases, addresses --

@pytest.mark.parametrize("R", [1, 16, 40, 300])
@pytest.mark.parametrize("fmt", FMTS)
def test_a_marked_block_makes_its_row_nan(R, fmt):
    N, K = 96, 1056
    x = _normal((R, K), 3)
    x[R // 2, K - 1] = np.inf
    c, s = qmoe.norm_act(fmt, to_gpu(x), torch.ones(K, device="cuda"), 1e-5)  # marks the block
    (Wg, Wu), _, _ = _real(fmt, 1, N, K, 5, pair=True)
    Wg, Wu = to_gpu(Wg), to_gpu(Wu)
    res = torch.zeros((R, N), device="cuda")
    for y in (qmoe.linear(fmt, Wg, N, K, c, s), qmoe.glu(fmt, Wg, Wu, N, K, c, s),
              qmoe.linear(fmt, Wg, N, K, c, s, act="relu", res=res, dtype=torch.bfloat16)):
        y = to_np(y.float())
        assert np.isnan(y[R // 2]).all()
        assert np.isfinite(np.delete(y, R // 2, axis=0)).all()
    q, d = (to_np(t) for t in qmoe.glu_act(fmt, Wg, Wu, N, K, c, s))
    bad = np.isnan(d) if fmt == "q8" else d == 255
    assert bad[R // 2].all() and not np.delete(bad, R // 2, axis=0).any()
    assert not q[R // 2].any()


@pytest.mark.parametrize("R,N", [(1, 33), (16, 130), (70, 132), (300, 264), (40, 31)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_residual_in_place_and_nothing_behind_the_last_row(R, N, fmt, bf):
    K = 288
    (W,), c, s = _real(fmt, R, N, K, 8)
    W, c, s = to_gpu(W), to_gpu(c), to_gpu(s)
    bias = to_gpu(_normal((1, N), 9)[0])
    big = torch.full((R + 3, N), 7.0, device="cuda", dtype=_dtype(bf))
    big[:R] = _dev(_normal((R, N), 10))
    want = qmoe.linear(fmt, W, N, K, c, s, bias=bias, act="silu", res=big[:R].clone(),
                       dtype=_dtype(bf))
    got = qmoe.linear(fmt, W, N, K, c, s, bias=bias, act="silu", res=big[:R], out=big[:R])
    assert got.data_ptr() == big.data_ptr()
    assert torch.equal(big[:R], want) and (big[R:] == 7.0).all()
    big.fill_(7.0)
    want = qmoe.glu(fmt, W, W, N, K, c, s, dtype=_dtype(bf))
    qmoe.glu(fmt, W, W, N, K, c, s, out=big[:R])     # the same weights twice
    assert torch.equal(big[:R], want) and (big[R:] == 7.0).all()


@pytest.mark.parametrize("R", [1, 16, 70, 300])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantized_output_behind_the_last_row(R, fmt):
    N, K = 160, 288
    (Wg, Wu), c, s = _real(fmt, R, N, K, 11, pair=True)
    args = (fmt, to_gpu(Wg), to_gpu(Wu), N, K, to_gpu(c), to_gpu(s))
    want = qmoe.glu_act(*args)
    big = [torch.full((R + 2,) + t.shape[1:], 77, dtype=t.dtype, device="cuda") for t in want]
    qmoe.glu_act(*args, out=(big[0][:R], big[1][:R]))
    for b, t in zip(big, want):
        assert torch.equal(b[:R], t) and (b[R:] == 77).all()


# int8 products: rows in one group of 16 and in several, and every tile, whose turn comes at
# these sizes on 256 units (linear's, then pairs')
@pytest.mark.parametrize("R,N", [(49, 535), (130, 2112), (300, 2016), (700, 2624), (1000, 3904),
                                 (2000, 4000), (100, 2080), (300, 2080), (520, 2080), (4, 26000),
                                 (13, 26000)])
def test_int8_choice_of_kernel(R, N):
    K = 416
    test_linear_on_an_exact_grid(R, N, K, "q8", True)
    test_glu_on_an_exact_grid(R, N, K, "q8", False)
    n = N // 32 * 32
    test_glu_quantized_is_the_quantizer_on_glu(R, n, K, "q8", "silu")
    for m in (N, N | 1):  # rows of whole pieces, and of any width
        test_residual_in_place_and_nothing_behind_the_last_row(R, m, "q8", True)
    (Wg, Wu), c, s = _real("q8", R, n, 288, 11, pair=True)
    args = ("q8", to_gpu(Wg), to_gpu(Wu), n, 288, to_gpu(c), to_gpu(s))
    want = qmoe.glu_act(*args)
    big = [torch.full((R + 2,) + t.shape[1:], 77, dtype=t.dtype, device="cuda") for t in want]
    qmoe.glu_act(*args, out=(big[0][:R], big[1][:R]))
    for b, t in zip(big, want):
        assert torch.equal(b[:R], t) and (b[R:] == 77).all()


@pytest.mark.parametrize("R,N,K", [(3, 70, 1056), (100, 130, 1056), (1200, 2100, 288)])
@pytest.mark.parametrize("fmt", FMTS)
def test_scales_and_bias_at_any_address(R, N, K, fmt):
    """E8M0 scales start at any byte, int8 scales and biases at any fp32."""
    (Wg, Wu), c, s = _real(fmt, R, N, K, 12, pair=True)
    Wg, Wu, c, s = to_gpu(Wg), to_gpu(Wu), to_gpu(c), to_gpu(s)
    bias = to_gpu(_normal((1, N), 13)[0])

    def odd(t):
        big = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        big[1:] = t.view(-1)
        assert big[1:].data_ptr() % 16
        return big[1:].view(t.shape)

    for f in (lambda c, s, b: qmoe.linear(fmt, Wg, N, K, c, s, bias=b, dtype=torch.bfloat16),
              lambda c, s, b: qmoe.glu(fmt, Wg, Wu, N, K, c, s, bias_gate=b, bias_up=b)):
        assert torch.equal(f(c, s, bias), f(c, odd(s), odd(bias)))


def test_empty_calls():
    z = lambda *sh, dt=torch.uint8: torch.zeros(sh, dtype=dt, device="cuda")
    for fmt in FMTS:
        ct, st = (torch.int8, torch.float32) if fmt == "q8" else (torch.uint8, torch.uint8)
        kc = 32 if fmt == "mxfp4" else 64
        W = z(qmoe.tensor_bytes(block.WEIGHTS[fmt], 32, 64))
        c, s = z(0, kc, dt=ct), z(0, 2, dt=st)
        assert qmoe.linear(fmt, W, 32, 64, c, s, res=z(0, 32, dt=torch.float32)).shape == (0, 32)
        assert qmoe.glu(fmt, W, W, 32, 64, c, s).shape == (0, 32)
        assert qmoe.glu_act(fmt, W, W, 32, 64, c, s)[1].shape == (0, 1)
        assert qmoe.linear(fmt, W, 0, 64, z(3, kc, dt=ct), z(3, 2, dt=st)).shape == (3, 0)
        x = z(0, 64, dt=torch.float32)
        w = z(64, dt=torch.float32)
        for gate in (None, w, x):
            assert qmoe.norm_block_act(fmt, x, x, w, 1e-5, gate=gate)[1].shape == (0, 2)
    assert qmoe.norm_block(x, x, w, 1e-5)[0].shape == (0, 64)


def _zeros_but_the_last(rows, last):
    big = torch.zeros((rows,) + last.shape[1:], dtype=last.dtype, device="cuda")
    big[rows - len(last):] = last
    return big


@pytest.mark.parametrize("fmt,R,N,K", [("mxfp8", 2, 2 ** 18 + 80, 32768), ("mxfp8", 2 ** 21 + 5, 48, 4096),
                                       ("mxfp8", 2 ** 26 + 5, 80, 32), ("q8", 2, 2 ** 17 + 80, 32768),
                                       ("q8", 40, 2 ** 17 + 80, 32768), ("q8", 2 ** 21 + 5, 48, 4096),
                                       ("q8", 2 ** 26 + 5, 80, 32), ("mxfp4", 40, 2 ** 18 + 80, 32768)])
def test_offsets_past_32_bits(fmt, R, N, K):
    """Weights, activations, residuals and outputs whose offsets pass 2^32, all of it
    zero but the last rows: sums there as in a call on those rows alone (exact, so in
    any order), and zeros elsewhere."""
    rng = np.random.default_rng(11)
    r, n = min(R, 40), min(N, 70)
    small = _grid_weights(rng, fmt, n, K)
    c, s = (to_gpu(t) for t in _grid_activations(rng, fmt, r, K))
    wf = block.WEIGHTS[fmt]
    small = to_gpu(small)
    want = qmoe.linear(fmt, small, n, K, c, s, dtype=torch.bfloat16)
    (c0, s0), (c1, s1) = qmoe.plane_offsets(wf, n, K), qmoe.plane_offsets(wf, N, K)
    W = torch.zeros(qmoe.tensor_bytes(wf, N, K), dtype=torch.uint8, device="cuda")
    per = (K, K // 16) if fmt == "q8" else (K // 2, K // 32)
    for row, o0, o1 in ((per[0], c0, c1), (per[1], s0, s1)):
        W[o1 + (N - n) * row:o1 + N * row] = small[o0:o0 + n * row]
    y = torch.ones((R, N), dtype=torch.bfloat16, device="cuda")
    c, s = _zeros_but_the_last(R, c), _zeros_but_the_last(R, s)
    qmoe.linear(fmt, W, N, K, c, s, res=y, out=y)
    assert torch.equal(y[R - r:, N - n:], qmoe.linear(
        fmt, small, n, K, c[R - r:].contiguous(), s[R - r:].contiguous(),
        res=torch.ones_like(want), dtype=torch.bfloat16))
    y[R - r:, N - n:] = 1
    assert (y == 1).all()
    del y
    if R * N < 2 ** 31:
        one = torch.ones(N, device="cuda")
        y = qmoe.glu(fmt, W, W, N, K, c, s, act=None, bias_up=one, dtype=torch.bfloat16)
        assert torch.equal(y[R - r:, N - n:], qmoe.glu(
            fmt, small, small, n, K, c[R - r:].contiguous(), s[R - r:].contiguous(), act=None,
            bias_up=one[:n], dtype=torch.bfloat16))
        y[R - r:, N - n:] = 0
        assert not y.any()


def test_sizes_past_31_bits_are_refused():
    u8 = dict(dtype=torch.uint8, device="cuda")
    for R, N, K in ((1, 2 ** 32 + 16, 32), (2 ** 32 + 1, 16, 32), (1, 16, 2 ** 32 + 64)):
        W = torch.empty((N * K // 2 + 511) // 256 * 256 + N * K // 32 + 512, **u8)
        c, s = torch.empty((R, K // 2), **u8), torch.empty((R, K // 32), **u8)
        with pytest.raises(qmoe.QmoeError):
            qmoe.linear("mxfp4", W, N, K, c, s, dtype=torch.bfloat16)
        with pytest.raises(qmoe.QmoeError):
            qmoe.glu("mxfp4", W, W, N, K, c, s, dtype=torch.bfloat16)


# ------------------------------------------------------------ norm block --

SIZES = [(1, 32), (1, 4096), (3, 96), (5, 2080), (300, 2048), (2, 7168), (3, 8224), (2, 16416),
         (1, 32768), (1100, 160), (1031, 8224), (4500, 32), (70, 64), (1000, 224), (9, 480),
         (600, 1568)]


def _check_stream(got, args, rbf, what):
    """h is the exact stream rounded, but where that is next to a border of two
    roundings: the kernel's fp64 value is within 2^-47 of its two terms' magnitudes.
    (A thread's 32 squares, 6 steps of a wave and 16 waves round the sum 54 times, the
    mean and eps twice, all halved by the root: 28 units of 2^-53; the root, the
    reciprocal, the products with the scale, the gate and x w_post, which is exact, and
    the last multiply-add add 7: below 2^-47.)  Rounding is monotone, so h lies between
    the roundings of the ends; one value of several millions is on another side."""
    exact, size = block.stream(*args)
    slack = size * np.longdouble(2.0) ** -47
    lo, hi = block.rounded(exact - slack, rbf), block.rounded(exact + slack, rbf)
    h = to_np(got.float())
    assert ((lo <= h) & (h <= hi)).all(), f"h {what}: {(~((lo <= h) & (h <= hi))).sum()} differ"
    assert (h != block.rounded(exact, rbf)).mean() < 1e-5
    return h


def _check_block(fmt, x, res, w, kw, xbf, rbf, what="", in_place=False):
    """h as above; codes and scales (or y) of that h bit for bit."""
    eps = 1e-5
    gate = kw.get("gate")
    gbf = gate is not None and (synth.bf16_round(gate) == gate).all()
    gk = dict(kw, w_post=_dev(kw.get("w_post")), gate=_dev(gate, gbf))
    gr = _dev(res, rbf)
    args = (_dev(x, xbf), gr, to_gpu(w), eps)
    if in_place:
        gk["res_out"] = gr
    if fmt in FMTS:
        q, s, gh = qmoe.norm_block_act(fmt, *args, **gk)
    else:
        got, gh = qmoe.norm_block(*args, dtype=_dtype(fmt == "bf16"), **gk)
    assert gh.dtype == _dtype(rbf) and (not in_place or gh is gr)
    h = _check_stream(gh, (x, res, kw.get("w_post"), kw.get("eps_post", eps), gate,
                           kw.get("scale", 1.0), kw.get("res_scale", 1.0)), rbf, what)
    y = act.rms_norm(h, w, eps)[0]
    if fmt in FMTS:
        wq, ws = act.quantize(fmt, y)
        assert (to_np(s) == ws).all(), f"{what}: {(to_np(s) != ws).sum()} scales differ"
        assert (to_np(q) == wq).all(), f"{what}: {(to_np(q) != wq).sum()} codes differ"
    else:
        assert_bitexact(to_np(got.float()), y if fmt == "f32" else act.bf16(y), what)


@pytest.mark.parametrize("R,K", SIZES)
@pytest.mark.parametrize("fmt", ("f32", "bf16") + FMTS)
def test_norm_block_sizes(R, K, fmt):
    x, res = _normal((R, K), 5), _normal((R, K), 6, 3.0, bf=True)
    w, wp = (1 + _normal((1, K), k, 0.1)[0] for k in (7, 8))
    gate = _normal((1, K), 9, bf=True)
    _check_block(fmt, x, res, w, dict(w_post=wp, gate=gate, scale=0.7, res_scale=1.25), False,
                 True, f"{fmt} {R}x{K}")


@pytest.mark.parametrize("xbf", [False, True], ids=["x_f32", "x_bf16"])
@pytest.mark.parametrize("rbf", [False, True], ids=["res_f32", "res_bf16"])
@pytest.mark.parametrize("post", [False, True], ids=["pre", "post"])
@pytest.mark.parametrize("gates", [0, 1, 3, -1])
@pytest.mark.parametrize("gbf", [False, True], ids=["gate_f32", "gate_bf16"])
def test_norm_block_types(xbf, rbf, post, gates, gbf):
    for R, K, fmt in ((6, 288, "mxfp8"), (1029, 288, "q8"), (9, 5216, "f32"), (1029, 4640, "mxfp4")):
        x, res = _normal((R, K), 10, bf=xbf), _normal((R, K), 11, 3.0, bf=rbf)
        kw = dict(scale=1.5, res_scale=0.75)
        if post:
            kw.update(w_post=1 + _normal((1, K), 12, 0.1)[0], eps_post=1e-3)
        if gates:
            kw["gate"] = _normal((R if gates < 0 else gates, K), 13, bf=gbf)
        w = 1 + _normal((1, K), 14, 0.1)[0]
        _check_block(fmt, x, res, w, kw, xbf, rbf, f"{R}x{K}", in_place=R == 6)


def test_norm_block_of_a_width_that_is_no_multiple_of_32():
    x, res, w = _normal((5, 1000), 15), _normal((5, 1000), 16), 1 + _normal((1, 1000), 17, 0.1)[0]
    _check_block("f32", x, res, w, dict(w_post=w), False, False)


def test_norm_block_without_its_additions_is_the_norm():
    x, res = to_gpu(_normal((40, 2080), 18)), to_gpu(_normal((40, 2080), 19))
    w = to_gpu(1 + _normal((1, 2080), 20, 0.1)[0])
    for fmt in FMTS:
        for a, b in zip(qmoe.norm_block_act(fmt, x, res, w, 1e-5),
                        qmoe.norm_act(fmt, x, w, 1e-5, res=res)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_block_zeros_huge_tiny_and_non_finite_rows(fmt):
    K = 256
    x, res = _normal((8, K), 21), _normal((8, K), 22)
    x[1], res[1] = 0.0, 0.0
    x[2] *= np.float32(1e30)       # squares beyond fp32
    x[3] *= np.float32(1e-30)      # squares below fp32
    x[4, 77] = np.nan
    res[5, 200] = np.inf
    w = np.ones(K, np.float32)
    fin = lambda a: np.where(np.isfinite(a), a, 0)
    y, h = block.norm_block(fin(x), fin(res), w, 1e-5, w, 1e-30)
    q, s, gh = (to_np(t) for t in qmoe.norm_block_act(fmt, to_gpu(x), to_gpu(res), to_gpu(w), 1e-5,
                                                      w_post=to_gpu(w), eps_post=1e-30))
    wq, ws = act.quantize(fmt, y)
    keep = [0, 1, 2, 3, 6, 7]
    assert (q[keep] == wq[keep]).all() and (s[keep] == ws[keep]).all()
    assert_bitexact(gh[keep], h[keep])
    bad = np.isnan(s) if fmt == "q8" else s == 255
    assert bad[4].all() and bad[5, 200 // 32] and not bad[keep].any()


def test_norm_block_of_one_tensor_in_every_place():
    """x, res and res_out are one tensor, and w_post is w."""
    x, w = _normal((40, 2080), 23), 1 + _normal((1, 2080), 24, 0.1)[0]
    g, gw = to_gpu(x), to_gpu(w)
    y, h = qmoe.norm_block(g, g, gw, 1e-5, w_post=gw, res_out=g)
    ry, rh = block.norm_block(x, x, w, 1e-5, w, 1e-5)
    assert h is g
    assert_bitexact(to_np(y), ry)
    assert_bitexact(to_np(g), rh)


def test_norm_block_offsets_past_32_bits_and_rows_behind():
    R, K, r = 2 ** 20 + 6, 4096, 6
    last = to_gpu(_normal((r, K), 25)).bfloat16()
    w = to_gpu(np.abs(_normal((1, K), 26)[0]))
    gate = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    gate[R - r:] = last
    x = gate.clone()
    for fmt in FMTS:
        got = qmoe.norm_block_act(fmt, x, x, w, 1e-5, w_post=w, gate=gate)
        want = qmoe.norm_block_act(fmt, last, last, w, 1e-5, w_post=w, gate=last)
        for a, b in zip(got, want):
            assert torch.equal(a[R - r:], b) and not a[:R - r].any()
    big = torch.full((r + 2, K), 7.0, device="cuda", dtype=torch.bfloat16)
    out = torch.full((r + 2, K), 7.0, device="cuda")
    qmoe.norm_block(last, last, w, 1e-5, res_out=big[:r], out=out[:r])
    assert (big[r:] == 7).all() and (out[r:] == 7).all()


# ---------------------------------------------------------- run together --

def _layer(fmt, x, res, P, H, F, act_name):
    """A sandwich-normed dense block as it is served: the norms behind the last block
    and before this one, gate and up, down, and the next pair of norms."""
    c, s, h = qmoe.norm_block_act(fmt, x, res, P["w"], 1e-5, w_post=P["wp"], gate=P["gate"],
                                  scale=0.7, res_scale=1.25)
    c2, s2 = qmoe.glu_act(fmt, P["Wg"], P["Wu"], F, H, c, s, act=act_name, bias_gate=P["bg"])
    d = qmoe.linear(fmt, P["Wd"], H, F, c2, s2, bias=P["bd"], dtype=torch.bfloat16)
    y, h2 = qmoe.norm_block(d, h, P["w"], 1e-5, w_post=P["wp"])
    z = qmoe.linear(fmt, P["Wd"], H, F, c2, s2, bias=P["bd"], res=h)     # a layer without post-norm
    return c, s, h, c2, s2, d, y, h2, z


def _params(fmt, H, F, seed):
    W = lambda n, k, i: to_gpu(fm.quantize(block.WEIGHTS[fmt],
                                           synth.normal((n, k), 0.05, seed, synth.GATE, i)))
    v = lambda n, k: to_gpu(1 + _normal((1, n), k, 0.1)[0])
    return dict(w=v(H, 1), wp=v(H, 2), gate=v(H, 3), bg=v(F, 4), bd=v(H, 5),
                Wg=W(F, H, 0), Wu=W(F, H, 1), Wd=W(H, F, 2))


@pytest.mark.parametrize("R", [1, 6, 16, 100, 600])
@pytest.mark.parametrize("fmt", FMTS)
def test_the_dense_block_run_together(R, fmt):
    """Every step against the oracle on that step's own inputs, and the whole run
    replayed as a graph, with eager calls in between."""
    H, F = 544, 1184
    P = _params(fmt, H, F, 3)
    x, res = to_gpu(_normal((R, H), 27)), to_gpu(_normal((R, H), 28, 2.0))
    out = _layer(fmt, x, res, P, H, F, "silu")
    c, s, h, c2, s2, d, y, h2, z = out
    p = {k: to_np(t) for k, t in P.items()}
    ry, rh = block.norm_block(to_np(x), to_np(res), p["w"], 1e-5, p["wp"], 1e-5, p["gate"], 0.7, 1.25)
    wq, ws = act.quantize(fmt, ry)
    assert (to_np(c) == wq).all() and (to_np(s) == ws).all()
    assert_bitexact(to_np(h), rh)
    g, ge = _sums(fmt, p["Wg"], F, H, wq, ws, False)
    u, ue = _sums(fmt, p["Wu"], F, H, wq, ws, False)
    f, fe = _activated("silu", g + p["bg"], ge + EPS * (np.abs(g) + np.abs(p["bg"])))
    err = fe * (np.abs(u) + ue) + np.abs(f) * ue
    err = err + EPS * (np.abs(f * u) + err)
    got = block.values(fmt, to_np(c2), to_np(s2)).reshape(R, -1, 32)
    v, err = (f * u).reshape(R, -1, 32), err.reshape(R, -1, 32)
    top = (np.abs(v) + err).max(-1, keepdims=True)
    # a code's rounding: int8 half a step of max / 127; E4M3 2^-4 of the value, an eighth
    # of it where it saturates, at least half of the smallest step; E2M1 a quarter of
    # the largest, where it saturates
    step = {"q8": top / 254 * 1.01, "mxfp8": np.abs(v) / 8 + top * 2.0 ** -17,
            "mxfp4": top / 4}[fmt]
    assert (np.abs(got - v) <= err * 1.13 + step * (1 + 2.0 ** -20)).all()
    v, e = _sums(fmt, p["Wd"], H, F, to_np(c2), to_np(s2), False)
    v, e = v + p["bd"], e + EPS * (np.abs(v) + np.abs(p["bd"]))
    _close(d, v, e, True)
    ry, rh = block.norm_block(to_np(d.float()), to_np(h), p["w"], 1e-5, p["wp"], 1e-5)
    assert_bitexact(to_np(y), ry)
    assert_bitexact(to_np(h2), rh)
    _close(z, v + to_np(h), e + EPS * (np.abs(v) + e + np.abs(to_np(h))), False)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = _layer(fmt, x, res, P, H, F, "silu")
    for seed in (29, 30, 31):
        x.copy_(to_gpu(_normal((R, H), seed)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, _layer(fmt, x, res, P, H, F, "silu")):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """No state is shared between calls: two streams at work together give what
    each gives alone."""
    H, F = 544, 1184
    runs = []
    for fmt, R in (("mxfp8", 9), ("q8", 300), ("mxfp4", 700)):
        P = _params(fmt, H, F, 4)
        x, res = to_gpu(_normal((R, H), R)), to_gpu(_normal((R, H), R + 1))
        runs.append(lambda fmt=fmt, P=P, x=x, res=res: _layer(fmt, x, res, P, H, F, "gelu"))
    want = [f() for f in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = [[] for _ in runs]
    for _ in range(4):
        for i, (st, f) in enumerate(zip(streams, runs)):
            with torch.cuda.stream(st):
                got[i].append(f())
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, w))
