"""The dense block's products over long K: every tile, and the few-row kernels, for many
turns of a team and a last one that ends inside a step."""
import numpy as np
import pytest

from gpu_util import requires_gpu, to_gpu, torch
from oracle import block
from oracle import formats as fm
from decode_moe_mul_amd import qmoe

pytestmark = [pytest.mark.gpu, requires_gpu]
F32, BF16 = torch.float32, torch.bfloat16

# (format, pair) -> (teams that split K, rows, columns) of every tile in the order of its
# list, whose turn comes at these sizes on 256 units
TILES = {
    ("mxfp4", False): [(4, 17, 32), (4, 610, 800), (2, 771, 1248), (2, 1604, 1184),
                       (1, 1667, 2336), (1, 2052, 3872)],
    ("mxfp8", False): [(4, 17, 32), (3, 610, 800), (2, 771, 1248), (1, 1156, 1696)],
    ("mxfp4", True): [(3, 17, 32), (2, 610, 800), (2, 771, 1248), (1, 1156, 1696),
                      (1, 1667, 3488)],
    ("mxfp8", True): [(3, 17, 32), (2, 610, 800), (1, 834, 1184)],
    ("q8", False): [(3, 421, 608), (2, 1156, 800), (1, 1793, 1056), (1, 1926, 3104)],
    ("q8", True): [(3, 435, 448), (2, 610, 800), (1, 834, 1184), (1, 1345, 2208)],
}
FEW = [(4, 3, 96), (4, 16, 160)]  # few rows: 16 waves split K
CASES = [(f, p, r, n, 4096 * t + 288) for (f, p), sizes in TILES.items()
         for t, r, n in sizes + FEW]
_SEPARATE = {"q8": qmoe.quantize_act_q8, "mxfp8": qmoe.quantize_act_mxfp8,
             "mxfp4": qmoe.quantize_act_mxfp4}
E4M3 = np.array([0, 0x30, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4A, 0x4C, 0x50, 0x52, 0x57], np.uint8)


def _operands(rng, fmt, R, N, K, pair):
    """Codes and scales of few binary places: every product is a multiple of 2^-4 (int8
    2^-2), and scales differ from block to block."""
    nb, W = K // 32, []
    for _ in range(2 if pair else 1):
        if fmt == "q8":
            W.append(fm.pack("q8_0", {
                "q": rng.integers(-12, 13, (N, nb, 32), dtype=np.int8),
                "d": (2.0 ** rng.integers(-1, 2, (N, nb))).astype(np.float16)}, N, K))
        else:
            W.append(fm.pack("mxfp4", {"q": rng.integers(0, 16, (N, K), dtype=np.uint8),
                                       "e": rng.integers(126, 129, (N, nb), dtype=np.uint8)},
                             N, K))
    if fmt == "q8":
        return W, rng.integers(-12, 13, (R, K), dtype=np.int8), \
            (2.0 ** rng.integers(-1, 2, (R, nb))).astype(np.float32)
    s = rng.integers(126, 129, (R, nb), dtype=np.uint8)
    if fmt == "mxfp4":
        return W, rng.integers(0, 256, (R, K // 2), dtype=np.uint8), s
    return W, E4M3[rng.integers(0, len(E4M3), (R, K))] | rng.integers(0, 2, (R, K),
                                                                      dtype=np.uint8) << 7, s


@pytest.mark.parametrize("fmt,pair,R,N,K", CASES)
def test_products_over_many_turns(fmt, pair, R, N, K):
    """Sums of magnitudes below 2^20 (int8 2^22): any order gives them to the bit, torch's
    product in fp32 too."""
    rng = np.random.default_rng(R + N + K)
    W, c, s = _operands(rng, fmt, R, N, K, pair)
    x = to_gpu(block.values(fmt, c, s).astype(np.float32))
    w = [to_gpu(fm.dequantize(block.WEIGHTS[fmt], v, N, K).astype(np.float32)) for v in W]
    assert (x.abs() @ w[0].abs().t()).max() < 2.0 ** (22 if fmt == "q8" else 20)
    sums = [x @ v.t() for v in w]
    W, c, s = [to_gpu(v) for v in W], to_gpu(c), to_gpu(s)
    # the same in 64 bits for the last rows and columns
    r, n = min(R, 5), min(N, 9)
    want = x[R - r:].double() @ w[0][N - n:].double().t()
    assert torch.equal(sums[0][R - r:, N - n:].double(), want)
    del x, w
    if not pair:
        assert torch.equal(qmoe.linear(fmt, W[0], N, K, c, s), sums[0])
        assert torch.equal(qmoe.linear(fmt, W[0], N, K, c, s, dtype=BF16), sums[0].bfloat16())
        return
    y = sums[0] * sums[1]
    assert torch.equal(qmoe.glu(fmt, *W, N, K, c, s, act=None), y)
    assert torch.equal(qmoe.glu(fmt, *W, N, K, c, s, act=None, dtype=BF16), y.bfloat16())
    for got, want in zip(qmoe.glu_act(fmt, *W, N, K, c, s, act=None), _SEPARATE[fmt](y)):
        assert torch.equal(got, want)
