"""The MXFP4 x MXFP4 product against the oracle, and the dense 4-bit MLP run
together."""
import numpy as np
import pytest

from gpu_util import requires_gpu, to_gpu, to_np, assert_bitexact, assert_within_bound, torch
from oracle import act
from oracle import formats as fm
from decode_moe_mul_amd import qmoe, synth

pytestmark = [pytest.mark.gpu, requires_gpu]

# rows around every kernel's tile, widths that end inside one, K of one block,
# K that ends inside a step of 128 and inside a turn of 512
SHAPES = [(1, 16, 32), (1, 1, 64), (1, 4096, 4096), (2, 49, 6752), (15, 130, 416), (16, 256, 512),
          (17, 33, 1056), (33, 640, 2048), (64, 2048, 640), (65, 100, 544), (130, 258, 1120),
          (257, 384, 224), (300, 515, 7200), (513, 1030, 160), (5, 9001, 288),
          # one of each tile size, odd and even numbers of steps, one step
          (300, 2001, 1312), (700, 2600, 352), (1000, 3900, 544), (2000, 4003, 800),
          (2040, 8100, 256), (2047, 8101, 1056)]


def _codes(rng, rows, K):
    return rng.integers(0, 16, (rows, K)).astype(np.uint8)


def _w(wc, we, N, K):
    return fm.pack("mxfp4", {"q": wc, "e": we}, N, K)


@pytest.mark.parametrize("R,N,K", SHAPES)
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_exact_grid(R, N, K, bf):
    """Scales of 1/2, 1 and 2: products are multiples of 1/16 and at most 144,
    sums below 2^20 in magnitude (K <= 7200), so every partial sum is exact in
    fp32 and any order of summation gives the oracle's value; a wrong pairing
    of values, blocks or scales changes it."""
    rng = np.random.default_rng(R * 7 + N + K)
    q, wq = _codes(rng, R, K), _codes(rng, N, K)
    e, we = (rng.integers(126, 129, (n, K // 32)).astype(np.uint8) for n in (R, N))
    buf = _w(wq, we, N, K)
    y = qmoe.gemm_mxfp4_mxfp4(to_gpu(buf), N, K, to_gpu(act.pack_codes(q)), to_gpu(e),
                              dtype=torch.bfloat16 if bf else None)
    ref, _ = act.gemm_mxfp4(buf, N, K, q, e)
    assert np.abs(ref).max() < 2 ** 20
    assert_bitexact(to_np(y.float()), act.bf16(ref.astype(np.float32)) if bf else ref)


@pytest.mark.parametrize("R,N,K", SHAPES)
def test_random_values(R, N, K):
    """fp32 sums of exact products in any order are within K 2^-24 sum |w x|."""
    x = synth.normal((R, K), 1.0, 3, synth.ACT, R) * np.exp2(
        np.random.default_rng(1).integers(-6, 6, (R, 1))).astype(np.float32)
    W = to_gpu(synth.normal((N, K), 0.02, 5, synth.GATE, 0))
    buf = qmoe.quantize("mxfp4", W)
    y = qmoe.gemm_mxfp4_mxfp4(buf, N, K, *qmoe.quantize_act_mxfp4(to_gpu(x)))
    ref, bound = act.gemm_mxfp4(to_np(buf), N, K, *act.quantize_mxfp4(x))
    assert_within_bound(to_np(y), ref, bound, rel=K * 2.0 ** -24, what=f"{R}x{N}x{K}")


@pytest.mark.parametrize("R", [1, 16, 40, 300])
def test_a_marked_block_makes_its_row_nan(R):
    N, K = 96, 1056
    x = synth.normal((R, K), 1.0, 3, synth.ACT, R)
    x[R // 2, K - 1] = np.inf
    W = qmoe.quantize("mxfp4", to_gpu(synth.normal((N, K), 0.02, 5, synth.GATE, 0)))
    y = to_np(qmoe.gemm_mxfp4_mxfp4(W, N, K, *qmoe.quantize_act_mxfp4(to_gpu(x))))
    assert np.isnan(y[R // 2]).all()
    assert np.isfinite(np.delete(y, R // 2, axis=0)).all()


@pytest.mark.parametrize("R", [1, 20, 300])
def test_extreme_scales(R):
    """Scale bytes 0 and 254 meet their opposites: products of 2^-127 x 2^127
    sized values are ordinary numbers."""
    N, K = 40, 256
    rng = np.random.default_rng(3)
    q, wq = _codes(rng, R, K), _codes(rng, N, K)
    lo = rng.integers(0, 2, (1, K // 32)) * 254
    e = np.repeat(lo, R, 0).astype(np.uint8)
    we = np.repeat(254 - lo, N, 0).astype(np.uint8)
    buf = _w(wq, we, N, K)
    y = qmoe.gemm_mxfp4_mxfp4(to_gpu(buf), N, K, to_gpu(act.pack_codes(q)), to_gpu(e))
    ref, _ = act.gemm_mxfp4(buf, N, K, q, e)
    assert_bitexact(to_np(y), ref)


@pytest.mark.parametrize("R,N", [(1, 40), (20, 40), (300, 40), (2100, 8100)])
@pytest.mark.parametrize("e", [57, 64, 70])
def test_products_and_sums_below_the_normal_numbers(R, N, e):
    """Scales of 2^-70 and less: every product is a multiple of 2^-142 and every sum
    below 2^-142 2^24, so all of them are fp32 numbers, most of them subnormal."""
    K = 256
    rng = np.random.default_rng(R + e)
    q, wq = _codes(rng, R, K), _codes(rng, N, K)
    buf = _w(wq, np.full((N, K // 32), 57, np.uint8), N, K)
    xe = np.full((R, K // 32), e, np.uint8)
    y = qmoe.gemm_mxfp4_mxfp4(to_gpu(buf), N, K, to_gpu(act.pack_codes(q)), to_gpu(xe))
    ref, bound = act.gemm_mxfp4(buf, N, K, q, xe)
    assert bound.max() < 2.0 ** (e - 57 - 142 + 24)
    assert_bitexact(to_np(y), ref)


@pytest.mark.parametrize("R,N", [(1, 33), (16, 130), (70, 130), (300, 258)])
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_nothing_is_written_behind_the_last_row(R, N, bf):
    K = 288
    W = qmoe.quantize("mxfp4", to_gpu(synth.normal((N, K), 0.02, 5, synth.GATE, 0)))
    c, s = qmoe.quantize_act_mxfp4(to_gpu(synth.normal((R, K), 1.0, 3, synth.ACT, R)))
    dt = torch.bfloat16 if bf else torch.float32
    big = torch.full((R + 3, N), 7.0, device="cuda", dtype=dt)
    qmoe.gemm_mxfp4_mxfp4(W, N, K, c, s, out=big[:R])
    assert (big[R:] == 7.0).all()
    assert torch.equal(big[:R], qmoe.gemm_mxfp4_mxfp4(W, N, K, c, s, dtype=dt))


@pytest.mark.parametrize("R,N,K", [(3, 70, 1056), (100, 130, 1056), (2040, 8100, 288)])
def test_scales_at_any_address(R, N, K):
    """Scale rows have K / 32 bytes and start anywhere: here at an odd address."""
    rng = np.random.default_rng(8)
    q, wq = _codes(rng, R, K), _codes(rng, N, K)
    e, we = (rng.integers(126, 129, (n, K // 32)).astype(np.uint8) for n in (R, N))
    W, codes = to_gpu(_w(wq, we, N, K)), to_gpu(act.pack_codes(q))
    want = qmoe.gemm_mxfp4_mxfp4(W, N, K, codes, to_gpu(e))
    odd = torch.zeros(e.size + 1, dtype=torch.uint8, device="cuda")
    odd[1:] = to_gpu(e).view(-1)
    scales = odd[1:].view(e.shape)
    assert scales.data_ptr() % 2 == 1
    assert torch.equal(want, qmoe.gemm_mxfp4_mxfp4(W, N, K, codes, scales))


def _zeros_but_the_last(rows, last):
    big = torch.zeros((rows,) + last.shape[1:], dtype=last.dtype, device="cuda")
    big[rows - len(last):] = last
    return big


@pytest.mark.parametrize("R,N,K", [(2, 2 ** 29 + 80, 32), (2 ** 21 + 5, 48, 4096),
                                   (2 ** 26 + 5, 80, 32)])
def test_offsets_past_32_bits(R, N, K):
    """Weights, activations and outputs whose offsets pass 2^32, all of it zero but
    the last rows: exact sums there, as in a call on those rows alone, and zeros
    elsewhere.  The widest W has more tiles of the smallest kind than a launch takes."""
    rng = np.random.default_rng(11)
    r, n = min(R, 40), min(N, 70)
    q, wq = _codes(rng, r, K), _codes(rng, n, K)
    e, we = (rng.integers(126, 129, (k, K // 32)).astype(np.uint8) for k in (r, n))
    small = to_gpu(_w(wq, we, n, K)), to_gpu(act.pack_codes(q)), to_gpu(e)
    want = qmoe.gemm_mxfp4_mxfp4(small[0], n, K, *small[1:], dtype=torch.bfloat16)
    (c0, s0), (c1, s1) = qmoe.plane_offsets("mxfp4", n, K), qmoe.plane_offsets("mxfp4", N, K)
    W = torch.zeros(qmoe.tensor_bytes("mxfp4", N, K), dtype=torch.uint8, device="cuda")
    for row, o0, o1 in ((K // 2, c0, c1), (K // 32, s0, s1)):
        W[o1 + (N - n) * row:o1 + N * row] = small[0][o0:o0 + n * row]
    y = torch.full((R, N), 3.0, dtype=torch.bfloat16, device="cuda")
    qmoe.gemm_mxfp4_mxfp4(W, N, K, _zeros_but_the_last(R, small[1]),
                          _zeros_but_the_last(R, small[2]), out=y)
    assert torch.equal(y[R - r:, N - n:], want)
    y[R - r:, N - n:] = 0
    assert not y.any()


@pytest.mark.parametrize("R,N,K", [(1, 2 ** 32 + 16, 32), (2 ** 32 + 1, 16, 32),
                                   (1, 16, 2 ** 32 + 64)])
def test_sizes_past_31_bits_are_refused(R, N, K):
    """The C entry takes sizes as 32-bit ints: a larger one is an error of the call,
    never its low bits.  The tensors are allocated only."""
    u8 = dict(dtype=torch.uint8, device="cuda")
    W = torch.empty(qmoe.tensor_bytes("mxfp4", 1, 32) + (N * K // 2 + 511) // 256 * 256
                    + N * K // 32, **u8)
    with pytest.raises(qmoe.QmoeError):
        qmoe.gemm_mxfp4_mxfp4(W, N, K, torch.empty((R, K // 2), **u8),
                              torch.empty((R, K // 32), **u8), dtype=torch.bfloat16)


def test_calls_on_two_streams_at_once():
    """No state is shared between calls: two streams at work together give what
    each gives alone."""
    N, K = 1030, 2080
    W = qmoe.quantize("mxfp4", to_gpu(synth.normal((N, K), 0.02, 5, synth.GATE, 0)))
    acts = [qmoe.quantize_act_mxfp4(to_gpu(synth.normal((R, K), 1.0, R, synth.ACT, R)))
            for R in (9, 700)]
    want = [qmoe.gemm_mxfp4_mxfp4(W, N, K, *a) for a in acts]
    streams = [torch.cuda.Stream() for _ in acts]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (st, a) in enumerate(zip(streams, acts)):
            with torch.cuda.stream(st):
                got[i].append(qmoe.gemm_mxfp4_mxfp4(W, N, K, *a))
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


def test_the_same_call_twice_gives_the_same_bits():
    """Two calls in turn give the same bits, and an empty one writes nothing."""
    N, K, R = 258, 1056, 270
    W = qmoe.quantize("mxfp4", to_gpu(synth.normal((N, K), 0.02, 5, synth.GATE, 0)))
    c, s = qmoe.quantize_act_mxfp4(to_gpu(synth.normal((R, K), 1.0, 3, synth.ACT, R)))
    a = qmoe.gemm_mxfp4_mxfp4(W, N, K, c, s)
    assert torch.equal(a, qmoe.gemm_mxfp4_mxfp4(W, N, K, c, s))
    assert qmoe.gemm_mxfp4_mxfp4(W, N, K, c[:0], s[:0]).shape == (0, N)


def _mlp(x, res, w, W, H, F):
    """One dense MLP with 4-bit operands: the chain as it is served."""
    c, s, h = qmoe.norm_act("mxfp4", x, w, 1e-5, res=res)
    gu = qmoe.gemm_mxfp4_mxfp4(W[0], 2 * F, H, c, s)
    c2, s2 = qmoe.swiglu_act("mxfp4", gu[:, :F], gu[:, F:])
    y = qmoe.gemm_mxfp4_mxfp4(W[1], H, F, c2, s2)
    n = qmoe.norm_act("mxfp8", y, w, 1e-5, res=h)
    return c, s, h, gu, c2, s2, y, n[0], n[1], n[2]


@pytest.mark.parametrize("R", [1, 6, 16, 100, 600])
def test_the_dense_mlp_run_together(R):
    """Every step against the oracle on that step's own inputs (products within
    K 2^-24 sum |w x|, everything else bit for bit), and the whole run
    replayed as a graph with eager calls in between."""
    H, F = 544, 1184
    x = to_gpu(synth.normal((R, H), 1.0, 1, synth.ACT, R))
    res = to_gpu(synth.normal((R, H), 2.0, 2, synth.ACT, R))
    w = to_gpu(1 + synth.normal((H,), 0.1, 3, synth.ACT, 0))
    W = [qmoe.quantize("mxfp4", to_gpu(synth.normal(sh, 0.05, 4, synth.GATE, i)))
         for i, sh in enumerate(((2 * F, H), (H, F)))]
    out = _mlp(x, res, w, W, H, F)
    c, s, h, gu, c2, s2, y, c3, s3, h3 = (to_np(t) for t in out)
    ry, rh = act.rms_norm(to_np(x), to_np(w), 1e-5, to_np(res))
    q, e = act.quantize_mxfp4(ry)
    assert (c == act.pack_codes(q)).all() and (s == e).all()
    assert_bitexact(h, rh)
    ref, bound = act.gemm_mxfp4(to_np(W[0]), 2 * F, H, q, e)
    assert_within_bound(gu, ref, bound, rel=H * 2.0 ** -24)
    q, e = act.quantize_mxfp4(act.swiglu(gu[:, :F], gu[:, F:]))
    assert (c2 == act.pack_codes(q)).all() and (s2 == e).all()
    ref, bound = act.gemm_mxfp4(to_np(W[1]), H, F, q, e)
    assert_within_bound(y, ref, bound, rel=F * 2.0 ** -24)
    ry, rh = act.rms_norm(y, to_np(w), 1e-5, h)
    want = act.quantize("mxfp8", ry)
    assert (c3 == want[0]).all() and (s3 == want[1]).all()
    assert_bitexact(h3, rh)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        held = _mlp(x, res, w, W, H, F)
    for seed in (5, 6, 7):
        x.copy_(to_gpu(synth.normal((R, H), 1.0, seed, synth.ACT, R)))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, _mlp(x, res, w, W, H, F)):
            assert torch.equal(a, b)
