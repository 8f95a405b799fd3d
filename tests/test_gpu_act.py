"""RMS norm with residual and quantized output, SwiGLU with quantized output,
the MXFP4 activation quantizer and its read-back: every output bit for bit
against the extended-precision oracle."""
import numpy as np
import pytest

from gpu_util import requires_gpu, to_gpu, to_np, assert_bitexact, torch
from oracle import act
from oracle import formats as fm
from decode_moe_mul_amd import qmoe, synth

pytestmark = [pytest.mark.gpu, requires_gpu]
FMTS = qmoe.ACT_FORMATS


def _x(shape, seed, sigma=1.0, bf=False):
    x = synth.normal(shape, sigma, seed, synth.ACT, shape[0])
    return synth.bf16_round(x) if bf else x


def _dev(x, bf):
    return to_gpu(x).to(torch.bfloat16) if bf else to_gpu(x)


def _same_act(got, want, what=""):
    q, s = to_np(got[0]), to_np(got[1])
    assert s.shape == want[1].shape and q.shape == want[0].shape
    same = (s == want[1]) | ((s != s) & (want[1] != want[1]))
    assert same.all(), f"{what}: {(~same).sum()} scales differ"
    assert (q == want[0]).all(), f"{what}: {(q != want[0]).sum()} code bytes differ"


# --------------------------------------------------------------- MXFP4 --

def _special():
    x = np.zeros((8, 64), np.float32)
    grid = fm.e2m1_value(np.arange(8))
    mids = (grid[:-1] + grid[1:]) / 2
    x[0, :8], x[0, 8:15], x[0, 15:22] = grid, mids, -mids      # every tie
    x[0, 32:] = -x[0, :32] * 2.0 ** -30
    x[1, :4] = [7.99, 6.5, 5.0, 7.0]                           # saturates at 6
    x[2] = -0.0
    x[3] = np.linspace(-3e-38, 3e-38, 64, dtype=np.float32)    # around the normal floor
    x[4] = np.float32(1e-45) * np.arange(64)                   # fp32 subnormals
    x[5, ::2] = 3.4e38
    x[6, 1] = np.nextafter(np.float32(4), np.float32(0))       # one step below a power of two
    x[7, 40] = 1e-30
    return x


def test_mxfp4_special_values():
    x = _special()
    _same_act(qmoe.quantize_act_mxfp4(to_gpu(x)), act.quantize("mxfp4", x))


def _signs():
    """Blocks whose negative values are zero in their block's scale: below half
    the element's smallest step, below fp32's smallest number, and -0, which is
    no negative value."""
    x = np.zeros((9, 64), np.float32)
    x[0, :3] = [1e30, -1e-30, -1e-45]
    x[1, :2] = [16, -1e-45]                       # -1e-45 / 2^E rounds to zero
    x[2, :2] = [4, -1e-45]                        # and is itself here (E = 0)
    x[3, :2] = [2.0 ** 100, -2.0 ** -60]
    x[4, :4] = [3.4e38, -1.2e-38, 1.2e-38, -0.0]
    x[5, :2] = [-1e30, 1e-30]
    x[6, 32:] = -1e-45
    x[6, 63] = 2.0 ** 127
    x[7] = -np.float32(2.0) ** -110
    x[7, ::32] = 2.0 ** 90
    x[8] = [(-1) ** k * np.float32(2.0) ** (7 * k // 2 - 110) for k in range(64)]
    return x


def test_the_sign_of_values_that_vanish_in_their_block():
    """Sign bit = (x < 0), as the weights' quantizer has it."""
    x = _signs()
    got = qmoe.quantize_act_mxfp4(to_gpu(x))
    want = act.quantize("mxfp4", x)
    assert want[0][0, 0] == 0x87                  # 1e30 saturates, -1e-30 is -0
    _same_act(got, want)
    W, off = qmoe.quantize("mxfp4", to_gpu(x)), qmoe.plane_offsets("mxfp4", *x.shape)
    assert torch.equal(got[0].view(-1), W[:x.size // 2])
    b = synth.bf16_round(x)
    _same_act(qmoe.quantize_act_mxfp4(_dev(b, True)), act.quantize("mxfp4", b))


@pytest.mark.parametrize("fmt", FMTS)
def test_the_sign_of_norm_and_swiglu_values_that_vanish_in_their_block(fmt):
    for w in _signs():
        x = np.ones((2, 64), np.float32)
        x[1] = -1                                 # y = w and -w: the mean square is 1
        y = act.rms_norm(x, w, 0.0)[0]
        assert (y[0] == w).all()
        _same_act(qmoe.norm_act(fmt, to_gpu(x), to_gpu(w), 0.0), act.quantize(fmt, y))
    u = _signs() / np.float32(64)                 # SwiGLU with a gate of 64 is 64 up
    g = np.full_like(u, 64)
    _same_act(qmoe.swiglu_act(fmt, to_gpu(g), to_gpu(u)), act.quantize(fmt, act.swiglu(g, u)))


@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (6, 2048), (5, 14336), (257, 160), (2, 65568)])
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
def test_mxfp4_quantizer_and_read_back(R, K, bf):
    x = _x((R, K), 3, bf=bf)
    got = qmoe.quantize_act_mxfp4(_dev(x, bf))
    want = act.quantize("mxfp4", x)
    _same_act(got, want)
    v = act.dequantize_mxfp4(*act.quantize_mxfp4(x))
    assert_bitexact(to_np(qmoe.dequantize_act_mxfp4(*got)), v)
    assert_bitexact(to_np(qmoe.dequantize_act_mxfp4(*got, dtype=torch.bfloat16).float()), v)


def test_mxfp4_codes_are_the_weights_quantizers():
    N, K = 33, 2048
    x = to_gpu(_x((N, K), 4, 0.02))
    codes, scales = qmoe.quantize_act_mxfp4(x)
    W, off = qmoe.quantize("mxfp4", x), qmoe.plane_offsets("mxfp4", N, K)
    assert torch.equal(codes.view(-1), W[:N * K // 2])
    assert torch.equal(scales.view(-1), W[off[1]:off[1] + N * K // 32])


def test_read_back_of_every_code_and_scale():
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    e = np.arange(256, dtype=np.uint8)[:, None]
    y = to_np(qmoe.dequantize_act_mxfp4(to_gpu(act.pack_codes(codes)), to_gpu(e)))
    with np.errstate(over="ignore"):
        assert_bitexact(y, act.dequantize_mxfp4(codes, e).astype(np.float32))


def test_bf16_read_back_of_every_code_and_scale():
    """bf16's subnormals, infinities and NaN among them: every finite value within
    bf16's range is exact."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    e = np.arange(256, dtype=np.uint8)[:, None]
    got = qmoe.dequantize_act_mxfp4(to_gpu(act.pack_codes(codes)), to_gpu(e),
                                    dtype=torch.bfloat16)
    with np.errstate(over="ignore"):              # 2^128 and above are infinite in both
        assert_bitexact(to_np(got.float()), act.dequantize_mxfp4(codes, e).astype(np.float32))


# ---------------------------------------------------------------- norm --

# one octet per thread, several waves a row, rows not a multiple of a block's,
# two and four octets per thread, several rows to a block in turn
SIZES = [(1, 32), (1, 4096), (3, 96), (5, 2080), (300, 2048), (2, 7168), (3, 8224), (2, 16416),
         (1, 32768), (1100, 160), (2100, 2080), (1031, 8224), (4500, 32),
         (70, 64), (1000, 224), (9, 480), (600, 7168)]


@pytest.mark.parametrize("R,K", SIZES)
@pytest.mark.parametrize("fmt", ("f32", "bf16") + FMTS)
def test_norm_sizes(R, K, fmt):
    x, res = _x((R, K), 5), _x((R, K), 6, 3.0, bf=True)
    w = 1 + _x((1, K), 7, 0.1)[0]
    y, h = act.rms_norm(x, w, 1e-5, res, res_bf16=True)
    gx, gw, gr = to_gpu(x), to_gpu(w), _dev(res, True)
    if fmt in FMTS:
        got = qmoe.norm_act(fmt, gx, gw, 1e-5, res=gr)
        _same_act(got, act.quantize(fmt, y), f"{fmt} {R}x{K}")
        gh = got[2]
    else:
        gy, gh = qmoe.norm(gx, gw, 1e-5, res=gr,
                           dtype=torch.float32 if fmt == "f32" else torch.bfloat16)
        assert_bitexact(to_np(gy.float()), y if fmt == "f32" else act.bf16(y))
    assert gh.dtype == torch.bfloat16
    assert_bitexact(to_np(gh.float()), h, "h")


@pytest.mark.parametrize("xbf", [False, True], ids=["x_f32", "x_bf16"])
@pytest.mark.parametrize("res", ["none", "f32", "bf16"])
@pytest.mark.parametrize("fmt", ("f32", "bf16") + FMTS)
def test_norm_types(xbf, res, fmt):
    for R, K in ((7, 288), (1027, 288)):
        x, r = _x((R, K), 8, bf=xbf), _x((R, K), 9, 3.0, bf=res == "bf16")
        w = 1 + _x((1, K), 7, 0.1)[0]
        gx, gw = _dev(x, xbf), to_gpu(w)
        gr = None if res == "none" else _dev(r, res == "bf16")
        y, h = act.rms_norm(x, w, 1e-6, None if res == "none" else r, res == "bf16")
        if fmt in FMTS:
            got = qmoe.norm_act(fmt, gx, gw, 1e-6, res=gr, res_out=gr)   # in place
            _same_act(got, act.quantize(fmt, y))
        else:
            dt = torch.float32 if fmt == "f32" else torch.bfloat16
            got = qmoe.norm(gx, gw, 1e-6, res=gr, res_out=gr, dtype=dt)
            got = got if gr is not None else (got,)
            assert_bitexact(to_np(got[0].float()), y if fmt == "f32" else act.bf16(y))
        if gr is not None:
            assert got[-1] is gr
            assert_bitexact(to_np(gr.float()), h)


def test_int8_codes_at_halves_and_with_tiny_scales():
    """Quotients on and next to k + 1/2, and scales down to the smallest
    subnormal: the block's largest value pins d."""
    k = np.arange(127, dtype=np.float32)
    v = np.concatenate([k + 0.5, np.nextafter(k + 0.5, 0), np.nextafter(k + 0.5, 200)])
    v = np.concatenate([v, -v]).astype(np.float32)
    v = np.concatenate([v, np.zeros(-len(v) % 31, np.float32)]).reshape(-1, 31)
    x = np.concatenate([np.full((len(v), 1), 127, np.float32), v], axis=1).reshape(1, -1)
    x = np.concatenate([x * np.float32(2.0) ** e for e in (0, 17, -60, -101, -126, -140)])
    x = np.pad(x, ((0, 0), (0, -x.shape[1] % 32)))
    # SwiGLU with a gate of 64 is 64 up, to fp32's last bit
    g, u = np.full_like(x, 64.0), x / np.float32(64.0)
    _same_act(qmoe.swiglu_act("q8", to_gpu(g), to_gpu(u)), act.quantize("q8", act.swiglu(g, u)))


_SEPARATE = {"q8": qmoe.quantize_act_q8, "mxfp8": qmoe.quantize_act_mxfp8,
             "mxfp4": qmoe.quantize_act_mxfp4}


@pytest.mark.parametrize("R,K", [(1, 4096), (16, 7168), (500, 2080)])
@pytest.mark.parametrize("fmt", FMTS)
def test_norm_then_quantizer_is_norm_act(fmt, R, K):
    """The fused call's codes and scales are those of the library's quantizer on
    the norm's fp32 rows, to the last bit of an int8 scale."""
    x, w = to_gpu(_x((R, K), 25)), to_gpu(1 + _x((1, K), 26, 0.1)[0])
    want = _SEPARATE[fmt](qmoe.norm(x, w, 1e-5))
    for a, b in zip(qmoe.norm_act(fmt, x, w, 1e-5), want):
        assert torch.equal(a, b)


def test_swiglu_then_int8_quantizer_is_swiglu_act():
    g, u = _x((200, 2080), 27, 1.5), _x((200, 2080), 28, 1.5)
    want = qmoe.quantize_act_q8(to_gpu(act.swiglu(g, u)))
    for a, b in zip(qmoe.swiglu_act("q8", to_gpu(g), to_gpu(u)), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("big", [1.0, 3e38, 2e-36, 1e-38, 1e-43, 1e-44, 2e-45], ids=str)
def test_int8_scale_of_any_size(big):
    """Block maxima of every size, fp32 subnormals and scales of zero among them."""
    x = (_x((4, 2048), 29) / 8).clip(-1, 1).astype(np.float32)
    x[:, ::32] = np.linspace(1, 0.25, 64, dtype=np.float32)
    x = (x * np.float32(big)).astype(np.float32)
    w = x[0].copy()                               # y = w: the mean square is 1
    ones = np.ones((1, 2048), np.float32)
    got = qmoe.norm_act("q8", to_gpu(ones), to_gpu(w), 0.0)
    want = act.quantize("q8", w[None])
    _same_act(got, want)
    for a, b in zip(got, qmoe.quantize_act_q8(to_gpu(w[None]))):
        assert torch.equal(a, b)


def test_int8_scale_of_every_significand():
    """One block for each fp32 significand as its maximum."""
    top = torch.arange(2 ** 23, dtype=torch.int32, device="cuda").add_(127 << 23).view(torch.float32)
    u = torch.zeros((2 ** 23, 32), device="cuda")
    u[:, 5] = top
    want = qmoe.quantize_act_q8(u)
    u.mul_(1 / 64)                                # SwiGLU with a gate of 64 is 64 up
    q, d = qmoe.swiglu_act("q8", torch.full_like(u, 64), u)
    assert torch.equal(d, want[1]) and torch.equal(q, want[0])


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_of_x_added_to_itself_in_place(fmt):
    """x, res and res_out are one tensor: h = 2 x."""
    x = _x((40, 2080), 22)
    w = np.ones(2080, np.float32)
    g = to_gpu(x)
    q, s, h = qmoe.norm_act(fmt, g, to_gpu(w), 1e-5, res=g, res_out=g)
    y, rh = act.rms_norm(x, w, 1e-5, x)
    _same_act((q, s), act.quantize(fmt, y))
    assert h is g
    assert_bitexact(to_np(g), rh)


def test_plain_norm_of_a_width_that_is_no_multiple_of_32():
    x, w = _x((5, 1000), 10), 1 + _x((1, 1000), 11, 0.1)[0]
    assert_bitexact(to_np(qmoe.norm(to_gpu(x), to_gpu(w), 1e-5)), act.rms_norm(x, w, 1e-5)[0])


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_rows_of_zeros_huge_tiny_and_non_finite_values(fmt):
    K = 256
    x = _x((8, K), 12)
    x[1] = 0.0
    x[2] *= np.float32(1e30)       # squares beyond fp32
    x[3] *= np.float32(1e-30)      # squares below fp32
    x[4, 77] = np.nan
    x[5, 200] = np.inf
    w = np.ones(K, np.float32)
    y = act.rms_norm(np.where(np.isfinite(x), x, 0), w, 1e-5)[0]
    y[4:6] = np.nan                # the row's norm is NaN or infinite: 0 or NaN times it
    q, s = (to_np(t) for t in qmoe.norm_act(fmt, to_gpu(x), to_gpu(w), 1e-5))
    wq, ws = act.quantize(fmt, y)
    keep = [0, 1, 2, 3, 6, 7]
    assert (q[keep] == wq[keep]).all() and (s[keep] == ws[keep]).all()
    bad = np.isnan(s) if fmt == "q8" else s == 255
    assert bad[4].all()
    assert bad[5, 200 // 32]       # inf * (1 / inf) is NaN; its neighbours are 0
    assert not bad[keep].any()


# -------------------------------------------------------------- SwiGLU --

@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (16, 14336), (130, 640), (1, 65536)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bf", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("joint", [False, True], ids=["separate", "halves"])
def test_swiglu(R, K, fmt, bf, joint):
    gu = _x((R, 2 * K), 13, 1.5, bf=bf)
    g, u = gu[:, :K], gu[:, K:]
    d = _dev(gu, bf)
    gg, uu = d[:, :K], d[:, K:]
    if not joint:
        gg, uu = gg.contiguous(), uu.contiguous()
    _same_act(qmoe.swiglu_act(fmt, gg, uu), act.quantize(fmt, act.swiglu(g, u)))


@pytest.mark.parametrize("fmt", FMTS)
def test_swiglu_far_values(fmt):
    g = np.zeros((4, 64), np.float32)
    g[0] = np.linspace(-120, 120, 64)
    g[1] = np.linspace(-3e38, 3e38, 64)
    g[2] = np.linspace(-1e-38, 1e-38, 64)
    g[3] = -np.linspace(80, 110, 64)
    u = np.where(np.arange(64) % 2, -1.0, 1.0).astype(np.float32) * np.ones((4, 1), np.float32)
    _same_act(qmoe.swiglu_act(fmt, to_gpu(g), to_gpu(u)), act.quantize(fmt, act.swiglu(g, u)))


@pytest.mark.parametrize("fmt", FMTS)
def test_swiglu_marks_non_finite_blocks(fmt):
    g, u = _x((3, 96), 14), _x((3, 96), 15)
    g[0, 3], u[1, 40], g[2, 95] = np.nan, np.inf, np.inf
    _, s = qmoe.swiglu_act(fmt, to_gpu(g), to_gpu(u))
    s = to_np(s)
    bad = np.isnan(s) if fmt == "q8" else s == 255
    want = np.zeros((3, 3), bool)
    want[0, 0] = want[1, 1] = want[2, 2] = True
    assert (bad == want).all()


# ------------------------------------------- streams, graphs, empty calls --

def test_empty_calls():
    x = torch.empty((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    assert qmoe.norm(x, w, 1e-5).shape == (0, 64)
    for fmt in FMTS:
        assert qmoe.norm_act(fmt, x, w, 1e-5, res=x)[1].shape == (0, 2)
        assert qmoe.swiglu_act(fmt, x, x)[1].shape == (0, 2)
    assert qmoe.dequantize_act_mxfp4(*qmoe.quantize_act_mxfp4(x)).shape == (0, 64)


def test_values_behind_the_last_row_stay():
    R, K = 3, 96
    x, w = to_gpu(_x((R, K), 16)), torch.ones(K, device="cuda")
    for fmt in FMTS:
        want = qmoe.norm_act(fmt, x, w, 1e-5)
        big = [torch.full((R + 2,) + t.shape[1:], 77, dtype=t.dtype, device="cuda") for t in want]
        qmoe.norm_act(fmt, x, w, 1e-5, out=(big[0][:R], big[1][:R]))
        for b, t in zip(big, want):
            assert torch.equal(b[:R], t) and (b[R:] == 77).all()


def test_offsets_past_32_bits():
    """More than 2^32 values: the last rows come out as in a call on them alone."""
    R, K, r = 2 ** 20 + 5, 4096, 7
    last = to_gpu(_x((r, 2 * K), 23)).bfloat16()
    w = to_gpu(np.abs(_x((K,), 24)))
    x = torch.zeros((R, 2 * K), dtype=torch.bfloat16, device="cuda")
    x[R - r:] = last
    for fmt in FMTS:
        got = qmoe.swiglu_act(fmt, x[:, :K], x[:, K:])
        for a, b in zip(got, qmoe.swiglu_act(fmt, last[:, :K], last[:, K:])):
            assert torch.equal(a[R - r:], b) and not a[:R - r].any()
    x, last = x[:, :K].contiguous(), last[:, :K].contiguous()
    for fmt in FMTS:
        got = qmoe.norm_act(fmt, x, w, 1e-5, res=x)
        for a, b in zip(got, qmoe.norm_act(fmt, last, w, 1e-5, res=last)):
            assert torch.equal(a[R - r:], b) and not a[:R - r].any()
    got, want = qmoe.quantize_act_mxfp4(x), qmoe.quantize_act_mxfp4(last)
    for a, b in zip(got, want):
        assert torch.equal(a[R - r:], b) and not a[:R - r].any()
    y = qmoe.dequantize_act_mxfp4(*got)
    assert torch.equal(y[R - r:], qmoe.dequantize_act_mxfp4(*want)) and not y[:R - r].any()


def test_sizes_past_31_bits_are_refused():
    """The C entries take rows as a 32-bit int: a larger count is an error of the
    call, never its low bits.  The tensors are allocated only."""
    R = 2 ** 32 + 5
    x = torch.empty((R, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(8, device="cuda")
    out = torch.empty((R, 8), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(qmoe.QmoeError):
        qmoe.norm(x, w, 1e-5, out=out)


def test_graph_replays_and_another_stream():
    R, K = 6, 2048
    x, res = to_gpu(_x((R, K), 17)), to_gpu(_x((R, K), 18))
    w = torch.ones(K, device="cuda")

    def step():
        c, s, h = qmoe.norm_act("mxfp4", x, w, 1e-5, res=res)
        c2, s2 = qmoe.swiglu_act("mxfp8", h, x)
        return c, s, h, c2, s2, qmoe.dequantize_act_mxfp4(c, s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(), [t.clone() for t in step()]):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (19, 20, 21):
        x.copy_(to_gpu(_x((R, K), seed)))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
