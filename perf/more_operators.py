"""What is measured of the dense block on quantized activations: the product with
bias, activation and residual in its epilogue, the gated pair of products with
the activation and the multiplication in one kernel, and the norms after and
before a block with its gate and residual scale between them.

``run`` computes a case in its plain form (elementary torch operations), or,
where ``own`` is true, by the library's calls.  Sizes are those of the
library's configurations (hidden widths 2048, 4096, 7168; FFN widths 640, 2048,
14336; 1, 6, 16 decode rows; 2048-row prefill chunks) and ragged ones between them.

Operands: "q8" is int8 activations with an fp32 scale per 32 values against Q8_0
weights, "mxfp8" and "mxfp4" are the MX activations against MXFP4 weights.
Outputs in MXFP8 are returned as the codes' E4M3 values and the scales' E8M0
values (views of the bytes), int8 ones as the integers with their fp32 scales,
MXFP4 ones read back as bfloat16 (every MXFP4 value is one).
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
_TORCH = {F32: torch.float32, BF16: torch.bfloat16}
_SIZE = {F32: 4, BF16: 2}
FORMATS = ("q8", "mxfp8", "mxfp4")
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu", "relu2")
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# bits of an activation and of a weight, with their scales
_BITS = {"q8": (9, 8.5), "mxfp8": (8.25, 4.25), "mxfp4": (4.25, 4.25)}


# ----------------------------------------------------------------- cases --

def listed():
    return [
        # one decoded token between two blocks: post-norm, scaled residual, the
        # next block's norm into an int8 product
        dict(name="norm_q8_1x4096", op="norm", out="q8", R=1, K=4096, x=F32, res=F32, post=True,
             gates=0, gate=F32),
        # 16 sessions' decode step, a gate row for every token
        dict(name="norm_mxfp4_16x7168", op="norm", out="mxfp4", R=16, K=7168, x=BF16, res=BF16,
             post=True, gates=16, gate=BF16),
        # four prefill chunks of the 7168-wide layer, gates per channel
        dict(name="norm_mxfp8_8192x7168", op="norm", out="mxfp8", R=8192, K=7168, x=BF16,
             res=BF16, post=True, gates=1, gate=F32),
        # one token's output projection added to the residual stream
        dict(name="linear_mxfp4_1x4096x4096", op="linear", fmt="mxfp4", R=1, N=4096, K=4096,
             y=F32, act="none", bias=False, res=F32),
        # 16 decode rows' down projection in int8, bf16 residual stream
        dict(name="linear_q8_16x4096x14336", op="linear", fmt="q8", R=16, N=4096, K=14336, y=BF16,
             act="none", bias=True, res=BF16),
        # a ragged batch through an ungated FFN's first product
        dict(name="linear_mxfp8_333x2050x7200", op="linear", fmt="mxfp8", R=333, N=2050, K=7200,
             y=BF16, act="gelu", bias=True, res="none"),
        # a prefill chunk's down projection with the residual
        dict(name="linear_mxfp4_2048x4096x14336", op="linear", fmt="mxfp4", R=2048, N=4096,
             K=14336, y=BF16, act="none", bias=False, res=BF16),
        # the 6 candidate rows of a speculative step, one narrow FFN
        dict(name="glu_mxfp8_6x640x2048", op="glu", fmt="mxfp8", R=6, N=640, K=2048, y=F32,
             act="silu", bias=False),
        # 16 decode rows, gate and up of the 14336-wide FFN
        dict(name="glu_mxfp4_16x14336x4096", op="glu", fmt="mxfp4", R=16, N=14336, K=4096, y=BF16,
             act="silu", bias=False),
        # a third of a chunk through a 2048-wide int8 FFN
        dict(name="glu_q8_700x2048x7168", op="glu", fmt="q8", R=700, N=2048, K=7168, y=BF16,
             act="silu", bias=True),
        # a prefill chunk, delivered in the down product's format
        dict(name="glu_mxfp8_2048x14336x4096", op="glu", fmt="mxfp8", R=2048, N=14336, K=4096,
             y="mxfp8", act="silu", bias=False),
        # the same with 4-bit activations, tanh-GELU, delivered in bf16
        dict(name="glu_mxfp4_2048x14336x4096", op="glu", fmt="mxfp4", R=2048, N=14336, K=4096,
             y=BF16, act="gelu_tanh", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "glu"))
    if op == "norm":
        K, x, res = 32 * _log(rng, 2, 448), rng.choice((F32, BF16)), rng.choice((F32, BF16))
        R = min(_log(rng, 1, 8192), 8192 * 7168 // K)
        R = max(1, R // 2) if F32 in (x, res) else R
        gates = rng.choice((0, 1, R, max(g for g in (1, 2, 3, 4, 5, 6, 7, 8) if R % g == 0)))
        gate = F32 if gates == 1 else rng.choice((F32, BF16))
        if gates == R and R > 1:
            R = gates = max(1, R // 2)
        return dict(op=op, out=rng.choice(FORMATS + (F32, BF16)), R=R, K=K, x=x, res=res,
                    post=rng.random() < 0.8, gates=gates, gate=gate)
    fmt, glu = rng.choice(FORMATS), op == "glu"
    most = 2048 * 14336 * 4096 // (8 if fmt == "q8" else 1) * (1 if glu else 2)
    R, N = _log(rng, 1, 2048), _log(rng, 32, 14336)
    K = 32 * _log(rng, 4, max(4, min(448, most // (32 * R * N))))
    act, bias = rng.choice(ACTS), rng.random() < 0.5
    if not glu:
        return dict(op=op, fmt=fmt, R=R, N=N, K=K, y=rng.choice((F32, BF16)), act=act, bias=bias,
                    res=rng.choice((F32, BF16, "none")))
    y = rng.choice((F32, BF16, "mxfp8" if fmt == "mxfp8" else BF16))
    return dict(op=op, fmt=fmt, R=R, N=N // 32 * 32 if y == "mxfp8" else N, K=K, y=y,
                act=rng.choice(("silu", act)), bias=bias)


# ---------------------------------------------------------------- inputs --

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, shape, dtype=torch.float32, sigma=1.0):
    return torch.randn(shape, generator=g, device=g.device).mul_(sigma).to(dtype)


def _mxfp4_bytes(v):
    """MXFP4 codes (two to a byte) and E8M0 bytes of v [rows, K]."""
    rows, K = v.shape
    q, e = _e2m1_block(v)
    lut = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], dtype=torch.uint8, device=v.device)
    codes = lut[(q.abs() * 2).to(torch.int64)] | ((v < 0).to(torch.uint8) << 3).view_as(q)
    codes = codes.view(rows, K // 2, 2)
    return (codes[..., 0] | (codes[..., 1] << 4)).contiguous(), e.to(torch.uint8)


def _activations(fmt, v):
    """(codes, scales) of v [R, K] as the library's quantizers lay them out."""
    if fmt == "mxfp4":
        return _mxfp4_bytes(v)
    if fmt == "mxfp8":
        got = _plain_mxfp8(v)
        return got["codes"].view(torch.uint8), got["scales"].view(torch.uint8)
    got = _plain_q8(v)
    return got["q"], got["d"]


def _weights(fmt, v):
    """Packed weights: all codes, then (256-byte aligned) all scales."""
    if fmt == "q8":
        got = _plain_q8(v)
        codes = got["q"].view(torch.uint8)
        scales = got["d"].to(torch.float16).view(torch.uint8)
    else:
        codes, scales = _mxfp4_bytes(v)
    n, at = codes.numel(), _scales_at(fmt, *v.shape)
    W = torch.zeros((at + scales.numel() + 255) // 256 * 256, dtype=torch.uint8, device=v.device)
    W[:n] = codes.view(-1)
    W[at:at + scales.numel()] = scales.view(-1)
    return W


def _scales_at(fmt, N, K):
    return (N * K // (1 if fmt == "q8" else 2) + 255) // 256 * 256


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(int(seed) * 1_000_003 + 29)
    c, st = case, {"case": case}
    R, K = c["R"], c["K"]
    if c["op"] == "norm":
        # a block's output with a few loud channels, and the stream it joins
        loud = 1.0 + 20.0 * (torch.rand(K, generator=g, device=g.device) < 0.005).float()
        st["x"] = (_normal(g, (R, K)) * loud).to(_TORCH[c["x"]])
        st["res"] = _normal(g, (R, K), _TORCH[c["res"]], 3.0)
        st["w"] = 1.0 + _normal(g, (K,), sigma=0.1)
        st["w_post"] = 1.0 + _normal(g, (K,), sigma=0.1) if c["post"] else None
        st["gate"] = None
        if c["gates"]:
            st["gate"] = torch.sigmoid(_normal(g, (c["gates"], K))).to(_TORCH[c["gate"]])
        st["scale"], st["res_scale"], st["eps"] = 0.7, 1.25, 1e-5
        return st
    N, fmt = c["N"], c["fmt"]
    for name in ("W",) if c["op"] == "linear" else ("Wg", "Wu"):
        st[name] = _weights(fmt, _normal(g, (N, K), sigma=0.02))
    st["codes"], st["scales"] = _activations(fmt, _normal(g, (R, K)))
    st["bias"] = _normal(g, (N,), sigma=0.5) if c["bias"] else None
    if c["op"] == "glu":
        st["bias_up"] = _normal(g, (N,), sigma=0.5) if c["bias"] else None
    else:
        st["res"] = None if c["res"] == "none" else _normal(g, (R, N), _TORCH[c["res"]], 3.0)
    return st


# ----------------------------------------------------------- plain forms --

def _two_to(e):
    """2^(e - 127) for integer tensors of E8M0 exponents in [0, 254]."""
    e = e.to(torch.int32)
    return torch.where(e == 0, 1 << 22, e << 23).to(torch.int32).view(torch.float32)


def _block_exponent(v, largest):
    """[rows, K/32, 32] blocks of v and their E8M0 exponents (floor of the
    base-2 logarithm of the block's largest magnitude, less `largest`)."""
    b = v.float().reshape(v.shape[0], v.shape[1] // 32, 32)
    amax = b.abs().amax(-1)
    ex = torch.frexp(amax).exponent.to(torch.int32) - 1
    return b, torch.where(amax > 0, (127 + ex - largest).clamp(0, 254), 0)


def _over_scale(b, e):
    # 2^-(e - 127) in two factors: one alone may leave fp32's range
    n = 127 - e
    h = n >> 1
    return (b * _two_to(h + 127)[..., None]) * _two_to(n - h + 127)[..., None]


def _e2m1_block(v):
    """E2M1 values of v / 2^E per block, shaped like v, and the exponents."""
    b, e = _block_exponent(v, 2)
    t = _over_scale(b, e)
    m = t.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    q = ((m / step).round() * step).clamp(max=6.0)
    return torch.copysign(q, t).view_as(v), e


def _plain_mxfp4(v):
    q, e = _e2m1_block(v)
    return (q.view(v.shape[0], -1, 32) * _two_to(e)[..., None]).view_as(v).to(torch.bfloat16)


def _plain_mxfp8(v):
    b, e = _block_exponent(v, 8)
    t = _over_scale(b, e)
    m = t.abs()
    # steps of 2^(floor(log2 m) - 3), at least 2^-9
    ex = (torch.frexp(m).exponent - 4).clamp(min=-9).to(torch.int32)
    q = ((m / _two_to(ex + 127)).round() * _two_to(ex + 127)).clamp(max=448.0)
    return {"codes": torch.copysign(q, t).view_as(v).to(torch.float8_e4m3fn),
            "scales": e.to(torch.uint8).view(torch.float8_e8m0fnu)}


def _plain_q8(v):
    b = v.reshape(v.shape[0], v.shape[1] // 32, 32)
    # a tensor divided by a tensor: by a Python number, torch multiplies by its reciprocal
    d = b.abs().amax(-1) / torch.full((), 127.0, device=v.device)
    r = torch.where(d[..., None] > 0, b / d[..., None], 0.0)
    t = r.trunc()
    q = (t + torch.where((r - t).abs() >= 0.5, r.sign(), 0.0)).clamp(-127, 127)
    return {"q": q.view_as(v).to(torch.int8), "d": d}


def _plain_out(out, v):
    if out in (F32, BF16):
        return {"y": v.to(_TORCH[out])}
    if out == "mxfp4":
        return {"y": _plain_mxfp4(v)}
    return _plain_mxfp8(v) if out == "mxfp8" else _plain_q8(v)


def _plain_fp4(codes, scales, rows):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    codes = codes.view(rows, -1).int()
    v = lut[torch.stack((codes & 15, codes >> 4), -1)].view(rows, -1, 32)
    return (v * _two_to(scales.view(rows, -1))[..., None]).view(rows, -1)


def _plain_weights(fmt, W, N, K):
    n, at = N * K // (1 if fmt == "q8" else 2), _scales_at(fmt, N, K)
    if fmt != "q8":
        return _plain_fp4(W[:n], W[at:at + N * K // 32], N)
    d = W[at:at + N * K // 16].view(torch.float16).float()
    return (W[:n].view(torch.int8).view(N, -1, 32).float() * d.view(N, -1, 1)).view(N, K)


def _plain_values(fmt, codes, scales):
    R = codes.shape[0]
    if fmt == "mxfp4":
        return _plain_fp4(codes, scales, R)
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float().view(R, -1, 32)
        return (v * _two_to(scales)[..., None]).view(R, -1)
    return (codes.view(R, -1, 32).float() * scales[..., None]).view(R, -1)


def _plain_act(act, v):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act in ("relu", "relu2"):
        p = torch.where(v > 0, v, 0.0)
        return p if act == "relu" else p * p
    return v


def _run_plain(st):
    c = st["case"]
    if c["op"] == "norm":
        # 64 bits up to the definition's roundings: codes next to a border
        z = st["x"].double()
        if st["w_post"] is not None:
            z = z * st["w_post"].double() / torch.sqrt(z.square().mean(-1, keepdim=True) + st["eps"])
        if st["gate"] is not None:
            z = (z.view(c["gates"], -1, c["K"]) * st["gate"].double()[:, None]).view_as(z)
        h = st["res_scale"] * st["res"].double() + st["scale"] * z
        h = h.float().to(st["res"].dtype)
        v = h.double()
        v = v * st["w"].double() / torch.sqrt(v.square().mean(-1, keepdim=True) + st["eps"])
        return {"h": h, **_plain_out(c["out"], v.float())}
    x = _plain_values(c["fmt"], st["codes"], st["scales"])
    if c["op"] == "linear":
        v = torch.matmul(x, _plain_weights(c["fmt"], st["W"], c["N"], c["K"]).t())
        v = _plain_act(c["act"], v if st["bias"] is None else v + st["bias"])
        v = v if st["res"] is None else v + st["res"].float()
        return {"y": v.to(_TORCH[c["y"]])}
    gate = torch.matmul(x, _plain_weights(c["fmt"], st["Wg"], c["N"], c["K"]).t())
    up = torch.matmul(x, _plain_weights(c["fmt"], st["Wu"], c["N"], c["K"]).t())
    if st["bias"] is not None:
        gate, up = gate + st["bias"], up + st["bias_up"]
    return _plain_out(c["y"], _plain_act(c["act"], gate) * up)


# ------------------------------------------------------- the library's calls --

def _own_out(out, pair):
    from decode_moe_mul_amd import qmoe

    if out == "mxfp4":
        return {"y": qmoe.dequantize_act_mxfp4(*pair, dtype=torch.bfloat16)}
    if out == "mxfp8":
        return {"codes": pair[0].view(torch.float8_e4m3fn),
                "scales": pair[1].view(torch.float8_e8m0fnu)}
    return {"q": pair[0], "d": pair[1]}


def _run_own(st):
    from decode_moe_mul_amd import qmoe

    c = st["case"]
    if c["op"] == "norm":
        more = dict(w_post=st["w_post"], gate=st["gate"], scale=st["scale"],
                    res_scale=st["res_scale"])
        if c["out"] in (F32, BF16):
            y, h = qmoe.norm_block(st["x"], st["res"], st["w"], st["eps"],
                                   dtype=_TORCH[c["out"]], **more)
            return {"h": h, "y": y}
        codes, scales, h = qmoe.norm_block_act(c["out"], st["x"], st["res"], st["w"], st["eps"],
                                               **more)
        return {"h": h, **_own_out(c["out"], (codes, scales))}
    act = None if c["act"] == "none" else c["act"]
    if c["op"] == "linear":
        return {"y": qmoe.linear(c["fmt"], st["W"], c["N"], c["K"], st["codes"], st["scales"],
                                 bias=st["bias"], act=act, res=st["res"], dtype=_TORCH[c["y"]])}
    args = (c["fmt"], st["Wg"], st["Wu"], c["N"], c["K"], st["codes"], st["scales"])
    more = dict(act=act, bias_gate=st["bias"], bias_up=st["bias_up"])
    if c["y"] in (F32, BF16):
        return {"y": qmoe.glu(*args, dtype=_TORCH[c["y"]], **more)}
    return _own_out(c["y"], qmoe.glu_act(*args, **more))


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    R, K = c["R"], c["K"]
    out = {"q8": 9 / 8, "mxfp8": 33 / 32, "mxfp4": 17 / 32 + 2, F32: 4, BF16: 2}
    if c["op"] == "norm":
        n = R * K * (_SIZE[c["x"]] + 2 * _SIZE[c["res"]] + out[c["out"]])
        n += c["gates"] * K * _SIZE[c["gate"]] + (8 if c["post"] else 4) * K
        return {"bytes": int(n), "flops": 14 * R * K}
    N, (xb, wb) = c["N"], _BITS[c["fmt"]]
    pair = 2 if c["op"] == "glu" else 1
    n = R * K * xb / 8 + pair * N * K * wb / 8 + R * N * out[c["y"]]
    n += 4 * N * pair * c["bias"] + (R * N * _SIZE.get(c.get("res"), 0))
    return {"bytes": int(n), "flops": 2 * pair * R * N * K}


# ------------------------------------------------------------------ exact --

def _nearest(v, grid):
    """The value of the sorted `grid` (from 0) nearest to |v|, the one with
    the even index on a tie, and v's sign."""
    m = v.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, m.contiguous()).clamp(1, grid.numel() - 1)
    a, b = grid[hi - 1], grid[hi]
    up = (b - m < m - a) | ((b - m == m - a) & (hi % 2 == 0))
    return torch.where(up, b, a) * v.sign()


def _exact_out(out, v):
    """What the format `out` holds of the values v, in 64 bits."""
    if out in (F32, BF16):
        return {"y": v}
    v = v.float().double()
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    if out == "q8":
        return {"q": None, "d": (amax / 127).squeeze(-1)}
    fp8 = out == "mxfp8"
    # floor(log2): the largest power of two not above amax
    p = torch.exp2(torch.log2(torch.where(amax > 0, amax, 1.0)).round())
    p = torch.where(p > amax, p / 2, p)
    p = torch.where(2 * p <= amax, 2 * p, p)
    s = torch.where(amax > 0, p / (256 if fp8 else 4), 2.0 ** -127).clamp(min=2.0 ** -127)
    if not fp8:
        grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
        return {"y": (_nearest(b / s, grid) * s).view_as(v)}
    # before its rounding, which either side takes: a code next to a border may
    # fall on either side of it
    return {"codes": (b / s).view_as(v), "scales": None}


def _exact_fp4(codes, scales, rows):
    scales = torch.exp2(scales.reshape(rows, -1).double() - 127)
    v = torch.empty((rows, scales.shape[1] * 32), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        k = (codes.reshape(rows, -1) >> (4 * half)) & 15
        mant, ex = (k & 1).double(), ((k >> 1) & 3).double()
        m = torch.where(ex == 0, mant / 2, (1 + mant / 2) * torch.exp2(ex - 1))
        v[:, half::2] = torch.where(k >= 8, -m, m)
    return v.mul_(scales.repeat_interleave(32, 1))


def _exact_weights(fmt, W, N, K):
    at = _scales_at(fmt, N, K)
    if fmt != "q8":
        return _exact_fp4(W[:N * K // 2], W[at:at + N * K // 32], N)
    d = W[at:at + N * K // 16].view(torch.float16).double().view(N, -1)
    return W[:N * K].view(torch.int8).double().view(N, K) * d.repeat_interleave(32, 1)


def _exact_values(fmt, codes, scales):
    R = codes.shape[0]
    if fmt == "mxfp4":
        return _exact_fp4(codes, scales, R)
    if fmt == "q8":
        return codes.double() * scales.double().repeat_interleave(32, 1)
    k = codes.to(torch.int64)
    ex, mant = (k >> 3) & 15, (k & 7).double()
    v = torch.where(ex == 0, mant * 2.0 ** -9, (1 + mant / 8) * torch.exp2(ex.double() - 7))
    v = torch.where(k >= 128, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _exact_act(act, v):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "relu":
        return v.clamp(min=0)
    return v.clamp(min=0) ** 2 if act == "relu2" else v


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        z = st["x"].double()
        if c["post"]:
            z = z * torch.rsqrt((z * z).sum(-1, keepdim=True) / c["K"] + st["eps"])
            z = z * st["w_post"].double()
        if c["gates"]:
            z = z * st["gate"].double().repeat_interleave(c["R"] // c["gates"], 0)
        total = st["res"].double() * st["res_scale"] + z * st["scale"]
        h = total.float().to(st["res"].dtype).double()
        v = h * torch.rsqrt((h * h).sum(-1, keepdim=True) / c["K"] + st["eps"]) * st["w"].double()
        return {"h": total, **_exact_out(c["out"], v)}
    fmt, N, K = c["fmt"], c["N"], c["K"]
    x = _exact_values(fmt, st["codes"], st["scales"])
    b = lambda v: 0.0 if v is None else v.double()
    if c["op"] == "linear":
        v = x @ _exact_weights(fmt, st["W"], N, K).t() + b(st["bias"])
        return {"y": _exact_act(c["act"], v) + b(st["res"])}
    gate = x @ _exact_weights(fmt, st["Wg"], N, K).t() + b(st["bias"])
    up = x @ _exact_weights(fmt, st["Wu"], N, K).t() + b(st["bias_up"])
    return _exact_out(c["y"], _exact_act(c["act"], gate) * up)
