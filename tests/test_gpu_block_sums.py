"""What the dense block's products keep of their sums: products far below the largest,
whatever the result's type and the kernel."""
import numpy as np
import pytest

from gpu_util import requires_gpu, to_gpu, to_np, assert_bitexact, torch
from oracle import act
from oracle import block
from oracle import formats as fm
from decode_moe_mul_amd import qmoe, synth

pytestmark = [pytest.mark.gpu, requires_gpu]
F32, BF16 = torch.float32, torch.bfloat16

# few rows, then a size for each tile of qlinear_mxfp8 and qglu_mxfp8 on 256 units
SHAPES = [(1, 40, 96), (3, 96, 1056), (16, 160, 2080), (17, 64, 544), (100, 130, 1056),
          (300, 2050, 288), (400, 4096, 288), (700, 2048, 288), (1000, 3900, 288)]


def _cancelling(rng, R, N, K, pair):
    """Eight consecutive values hold 448, -448 and six codes below 2, the weights of the
    two large ones are equal: a sum is that of the small products alone, multiples of
    2^-11 (2^-9 of a code, 2^-1 of a weight and of its scale) below 2^13: exact in fp32
    in any order, and nothing is left of it where a product 13 binary places below the
    largest is dropped."""
    c = (rng.integers(0, 64, (R, K)) | rng.integers(0, 2, (R, K)) << 7).astype(np.uint8)
    W = []
    g = np.arange(0, K, 8)
    p = rng.permuted(np.tile(np.arange(8), (g.size, 1)), axis=1)
    c[:, g + p[:, 0]], c[:, g + p[:, 1]] = 0x7E, 0xFE
    s = np.full((R, K // 32), 127, np.uint8)
    for _ in range(2 if pair else 1):
        q = rng.integers(0, 16, (N, K)).astype(np.uint8)
        q[:, g + p[:, 1]] = q[:, g + p[:, 0]]
        e = rng.integers(126, 129, (N, K // 32)).astype(np.uint8)
        W.append(fm.pack("mxfp4", {"q": q, "e": e}, N, K))
    low = c.copy()
    low[:, g + p[:, 0]], low[:, g + p[:, 1]] = 0, 0
    sums = []
    for w in W:
        y, b = block.product("mxfp8", w, N, K, low, s)
        assert b.max() < 2.0 ** 13 and np.count_nonzero(y)
        sums.append(y)
    return [to_gpu(w) for w in W], to_gpu(c), to_gpu(s), sums


@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_mxfp8_sums_of_small_products_beside_large_ones(R, N, K, dtype):
    rng = np.random.default_rng(R + N + K)
    W, c, s, (g, u) = _cancelling(rng, R, N, K, True)
    out = (lambda v: act.bf16(v)) if dtype is BF16 else lambda v: v
    for w, y in zip(W, (g, u)):
        got = qmoe.linear("mxfp8", w, N, K, c, s, dtype=dtype)
        assert_bitexact(to_np(got.float()), out(y.astype(np.float32)), "linear")
    got = qmoe.glu("mxfp8", *W, N, K, c, s, act=None, dtype=dtype)
    assert_bitexact(to_np(got.float()), out((g * u).astype(np.float32)), "pair")


@pytest.mark.parametrize("R,N,K", [(r, n // 32 * 32, k) for r, n, k in SHAPES])
def test_mxfp8_codes_of_small_products_beside_large_ones(R, N, K):
    rng = np.random.default_rng(R + N + K)
    W, c, s, (g, u) = _cancelling(rng, R, N, K, True)
    codes, scales = qmoe.glu_act("mxfp8", *W, N, K, c, s, act=None)
    wq, ws = act.quantize("mxfp8", (g * u).astype(np.float32))
    assert (to_np(scales) == ws).all() and (to_np(codes) == wq).all()


@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("fmt", qmoe.ACT_FORMATS)
def test_a_results_type_changes_its_rounding_alone(R, N, K, fmt):
    """Three channels a thousand times louder than the others."""
    x = synth.normal((R, K), 1.0, 3, synth.ACT, R)
    x[:, [1, K // 2 + 3, K - 7]] *= 1000
    c, s = (to_gpu(t) for t in act.quantize(fmt, x))
    Wg, Wu = (to_gpu(fm.quantize(block.WEIGHTS[fmt], synth.normal((N, K), 0.02, 3, synth.GATE, i)))
              for i in range(2))
    for f in (lambda d: qmoe.linear(fmt, Wg, N, K, c, s, dtype=d),
              lambda d: qmoe.glu(fmt, Wg, Wu, N, K, c, s, dtype=d)):
        assert torch.equal(f(F32).bfloat16(), f(BF16))


@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_mxfp8_sums_of_large_codes_are_exact(R, N, K, dtype):
    """Codes from 2 to 448, the largest beside the smallest: multiples of 2^-3 (2^-2 of a
    code, 2^-1 of a weight) below 2^21."""
    rng = np.random.default_rng(R + N + K)
    c = rng.integers(0x40, 0x7F, (R, K)).astype(np.uint8)
    c[:, ::8], c[:, 3::8] = 0x7E, 0x41
    c |= (rng.integers(0, 2, (R, K)) << 7).astype(np.uint8)
    s = np.full((R, K // 32), 127, np.uint8)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    q[:, ::8], q[:, 3::8] = 7, 1
    W = fm.pack("mxfp4", {"q": q, "e": np.full((N, K // 32), 127, np.uint8)}, N, K)
    y, b = block.product("mxfp8", W, N, K, c, s)
    assert b.max() < 2.0 ** 21
    got = qmoe.linear("mxfp8", to_gpu(W), N, K, to_gpu(c), to_gpu(s), dtype=dtype)
    y = y.astype(np.float32)
    assert_bitexact(to_np(got.float()), act.bf16(y) if dtype is BF16 else y)
