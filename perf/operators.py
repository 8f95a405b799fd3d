"""What is measured of the quantized-activation operators: the RMS norm with
the residual's addition and a quantized output, the MXFP4 quantizer of
activations and its read-back, SwiGLU with a quantized output, and the
MXFP4 x MXFP4 product.

``run`` computes a case in its plain form (elementary torch operations), or,
where ``own`` is true, by the library's calls.  Sizes are those of the
library's configurations (hidden widths 2048, 4096, 7168; FFN width 14336;
1, 6, 16 decode rows; 2048-row prefill chunks) and ragged ones between them.

Outputs: MXFP8 results are returned as the codes' E4M3 values and the scales'
E8M0 values (views of the bytes), int8 results as the integers with their fp32
scales, MXFP4 results read back as bfloat16 (every MXFP4 value is one).
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
_TORCH = {F32: torch.float32, BF16: torch.bfloat16}
_SIZE = {F32: 4, BF16: 2}
NORM_OUT = ("q8", "mxfp8", "mxfp4", "bf16", "f32")
ACT_OUT = ("q8", "mxfp8", "mxfp4")
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- cases --

def listed():
    return [
        # one decoded token's residual stream into an int8 product (4096-wide layer)
        dict(name="norm_q8_1x4096", op="norm", out="q8", R=1, K=4096, x=F32, res=F32),
        # 16 sessions' decode step, 7168-wide, into a 4-bit product
        dict(name="norm_mxfp4_16x7168", op="norm", out="mxfp4", R=16, K=7168, x=BF16, res=BF16),
        # one prefill chunk of the 2048-wide layer; products deliver fp32
        dict(name="norm_mxfp8_2048x2048", op="norm", out="mxfp8", R=2048, K=2048, x=F32, res=F32),
        # four prefill chunks of the 7168-wide layer, bf16 stream
        dict(name="norm_mxfp8_8192x7168", op="norm", out="mxfp8", R=8192, K=7168, x=BF16, res=BF16),
        # activations of a speculative step (6 candidate rows) to MXFP4 and back
        dict(name="mxfp4_6x2048", op="quant", R=6, K=2048, x=F32),
        # a chunk's FFN activations to MXFP4 and back
        dict(name="mxfp4_2048x14336", op="quant", R=2048, K=14336, x=BF16),
        # 16 decode rows between the gate/up and the down product, int8
        dict(name="swiglu_q8_16x14336", op="swiglu", out="q8", R=16, K=14336, x=F32, joint=True),
        # the same for a prefill chunk, MXFP4
        dict(name="swiglu_mxfp4_2048x14336", op="swiglu", out="mxfp4", R=2048, K=14336, x=BF16,
             joint=True),
        # one token against a square projection
        dict(name="gemm_1x4096x4096", op="gemm", R=1, N=4096, K=4096, y=F32),
        # 16 decode rows against gate or up
        dict(name="gemm_16x14336x4096", op="gemm", R=16, N=14336, K=4096, y=F32),
        # a ragged batch, no size a multiple of any tile
        dict(name="gemm_333x2050x7200", op="gemm", R=333, N=2050, K=7200, y=BF16),
        # a prefill chunk against gate or up
        dict(name="gemm_2048x14336x4096", op="gemm", R=2048, N=14336, K=4096, y=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "quant", "swiglu", "gemm", "gemm"))
    if op == "gemm":
        R, N = _log(rng, 1, 2048), _log(rng, 16, 14336)
        K = 32 * _log(rng, 4, min(448, 2048 * 14336 * 128 // (R * N)))
        return dict(op=op, R=R, N=N, K=K, y=rng.choice((F32, BF16)))
    K = 32 * _log(rng, 2, 448)
    R = _log(rng, 1, 8192)
    R = min(R, (8192 * 7168 if op == "norm" else 2048 * 14336) // K)
    x = rng.choice((F32, BF16))
    if op == "quant":
        return dict(op=op, R=R if x == BF16 else max(1, R // 2), K=K, x=x)
    if op == "swiglu":
        return dict(op=op, out=rng.choice(ACT_OUT), R=R if x == BF16 else max(1, R // 2), K=K,
                    x=x, joint=rng.random() < 0.7)
    res = rng.choice((F32, BF16, "none"))
    return dict(op=op, out=rng.choice(NORM_OUT), R=max(1, R // 2) if F32 in (x, res) else R, K=K,
                x=x, res=res)


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


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(int(seed) * 1_000_003 + 17)
    c, st = case, {"case": case}
    R, K = c["R"], c["K"]
    if c["op"] == "gemm":
        # weights as a checkpoint holds them: all codes, then (256-byte aligned) all scales
        wc, ws = _mxfp4_bytes(_normal(g, (c["N"], K), sigma=0.02))
        n = wc.numel()
        at = (n + 255) // 256 * 256
        W = torch.zeros((at + ws.numel() + 255) // 256 * 256, dtype=torch.uint8, device=g.device)
        W[:n] = wc.view(-1)
        W[at:at + ws.numel()] = ws.view(-1)
        st["W"], st["scales_at"] = W, at
        st["codes"], st["scales"] = _mxfp4_bytes(_normal(g, (R, K)))
    elif c["op"] == "norm":
        # a residual stream with a few loud channels, as trained layers have them
        loud = 1.0 + 20.0 * (torch.rand(K, generator=g, device=g.device) < 0.005).float()
        st["x"] = (_normal(g, (R, K)) * loud).to(_TORCH[c["x"]])
        st["res"] = None if c["res"] == "none" else _normal(g, (R, K), _TORCH[c["res"]], 3.0)
        st["w"] = 1.0 + _normal(g, (K,), sigma=0.1)
        st["eps"] = 1e-5
    elif c["op"] == "swiglu":
        if c["joint"]:   # the two halves of one product's rows
            gu = _normal(g, (R, 2 * K), _TORCH[c["x"]], 1.5)
            st["gate"], st["up"] = gu[:, :K], gu[:, K:]
        else:
            st["gate"] = _normal(g, (R, K), _TORCH[c["x"]], 1.5)
            st["up"] = _normal(g, (R, K), _TORCH[c["x"]], 1.5)
    else:
        st["x"] = _normal(g, (R, K), _TORCH[c["x"]])
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
    d = b.abs().amax(-1) / 127
    r = torch.where(d[..., None] > 0, b / d[..., None], 0.0)
    t = r.trunc()
    q = (t + torch.where((r - t).abs() >= 0.5, r.sign(), 0.0)).clamp(-127, 127)
    return {"q": q.view_as(v).to(torch.int8), "d": d}


def _plain_act(out, v):
    if out in (F32, BF16):
        return {"y": v.to(_TORCH[out])}
    if out == "mxfp4":
        return {"y": _plain_mxfp4(v)}
    return _plain_mxfp8(v) if out == "mxfp8" else _plain_q8(v)


def _run_plain(st):
    c = st["case"]
    if c["op"] == "gemm":
        R, N, K = c["R"], c["N"], c["K"]
        n, at = N * K // 2, st["scales_at"]
        lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=st["W"].device)

        def values(codes, scales, rows):
            codes = codes.view(rows, K // 2).int()
            v = lut[torch.stack((codes & 15, codes >> 4), -1)].view(rows, K // 32, 32)
            return (v * _two_to(scales.view(rows, K // 32))[..., None]).view(rows, K)

        w = values(st["W"][:n], st["W"][at:at + N * K // 32], N)
        x = values(st["codes"], st["scales"], R)
        return {"y": torch.matmul(x, w.t()).to(_TORCH[c["y"]])}
    if c["op"] == "quant":
        return {"y": _plain_mxfp4(st["x"].float())}
    if c["op"] == "swiglu":
        # 64 bits up to the definition's one rounding: codes next to a border
        g = st["gate"].double()
        return _plain_act(c["out"], (g / (1 + torch.exp(-g)) * st["up"].double()).float())
    h = st["x"]
    if st["res"] is not None:
        h = (h.float() + st["res"].float()).to(st["res"].dtype)
    v = h.double()
    v = v * st["w"].double() / torch.sqrt(v.square().mean(-1, keepdim=True) + st["eps"])
    got = _plain_act(c["out"], v.float())
    return {"h": h, **got} if st["res"] is not None else got


# ------------------------------------------------------- the library's calls --

def _own_act(out, pair):
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
    if c["op"] == "gemm":
        return {"y": qmoe.gemm_mxfp4_mxfp4(st["W"], c["N"], c["K"], st["codes"], st["scales"],
                                           dtype=_TORCH[c["y"]])}
    if c["op"] == "quant":
        return _own_act("mxfp4", qmoe.quantize_act_mxfp4(st["x"]))
    if c["op"] == "swiglu":
        return _own_act(c["out"], qmoe.swiglu_act(c["out"], st["gate"], st["up"]))
    if c["out"] in (F32, BF16):
        got = qmoe.norm(st["x"], st["w"], st["eps"], res=st["res"], dtype=_TORCH[c["out"]])
        return {"y": got[0], "h": got[1]} if st["res"] is not None else {"y": got}
    got = qmoe.norm_act(c["out"], st["x"], st["w"], st["eps"], res=st["res"])
    act = _own_act(c["out"], got[:2])
    return {"h": got[2], **act} if st["res"] is not None else act


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    R, K = c["R"], c["K"]
    if c["op"] == "gemm":
        N = c["N"]
        return {"bytes": (N + R) * K * 17 // 32 + R * N * _SIZE[c["y"]], "flops": 2 * R * N * K}
    # per value: codes and scales, and for MXFP4 the values read back from them
    out = {"q8": 1 + 4 / 32, "mxfp8": 1 + 1 / 32, "mxfp4": 17 / 32 + 2, F32: 4, BF16: 2}
    if c["op"] == "quant":
        return {"bytes": R * K * (_SIZE[c["x"]] + out["mxfp4"]), "flops": 4 * R * K}
    if c["op"] == "swiglu":
        return {"bytes": R * K * (2 * _SIZE[c["x"]] + out[c["out"]]), "flops": 8 * R * K}
    res = 0 if c["res"] == "none" else 2 * _SIZE[c["res"]]
    return {"bytes": R * K * (_SIZE[c["x"]] + res + out[c["out"]]) + 4 * K, "flops": 8 * R * K}


# ------------------------------------------------------------------ exact --

def _nearest(v, grid):
    """The value of the sorted `grid` (from 0) nearest to |v|, the one with
    the even index on a tie, and v's sign."""
    m = v.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, m.contiguous()).clamp(1, grid.numel() - 1)
    a, b = grid[hi - 1], grid[hi]
    up = (b - m < m - a) | ((b - m == m - a) & (hi % 2 == 0))
    return torch.where(up, b, a) * v.sign()


def _exact_act(out, v):
    """What the format `out` holds of the fp32 values v, in 64 bits."""
    v = v.double()
    if out in (F32, BF16):
        return {"y": v}
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
    grid = [m / 8 * 2.0 ** -6 for m in range(8)]
    grid += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    return {"codes": _nearest(b / s, grid).view_as(v), "scales": s.squeeze(-1)}


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "gemm":
        K = c["K"]

        def values(codes, scales, rows):
            scales = torch.exp2(scales.reshape(rows, -1).double() - 127)
            v = torch.empty((rows, K), dtype=torch.float64, device=codes.device)
            for half in (0, 1):
                k = (codes.reshape(rows, -1) >> (4 * half)) & 15
                mant, ex = (k & 1).double(), ((k >> 1) & 3).double()
                m = torch.where(ex == 0, mant / 2, (1 + mant / 2) * torch.exp2(ex - 1))
                v[:, half::2] = torch.where(k >= 8, -m, m)
            return v * scales.repeat_interleave(32, 1)

        at = st["scales_at"]
        w = values(st["W"][:c["N"] * K // 2], st["W"][at:at + c["N"] * K // 32], c["N"])
        return {"y": values(st["codes"], st["scales"], c["R"]) @ w.t().contiguous()}
    if c["op"] == "quant":
        return _exact_act("mxfp4", st["x"])
    if c["op"] == "swiglu":
        g, u = st["gate"].double(), st["up"].double()
        return _exact_act(c["out"], (g * u * torch.sigmoid(g)).float())
    if st["res"] is None:
        h = st["x"].double()
    else:
        total = st["x"].double() + st["res"].double()
        h = total.float().to(st["res"].dtype).double()  # the fp32 sum, rounded to its type
    v = h * torch.rsqrt((h * h).sum(-1, keepdim=True) / c["K"] + st["eps"]) * st["w"].double()
    got = _exact_act(c["out"], v if c["out"] in (F32, BF16) else v.float())
    return got if st["res"] is None else {"h": total, **got}
