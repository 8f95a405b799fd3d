"""Thin Python binding of libqmoe.so (include/qmoe.h).

Argument marshalling only: every step runs in the HIP kernels of the library.
Tensors are torch tensors on the GPU (PyTorch supplies device memory and the
current stream); the functions allocate outputs and workspaces with torch and
pass raw pointers.  If the library is missing, the first call raises -- there
is no fallback path.
"""
import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqmoe.so")

FORMATS = {"q8_0": 0, "q4_0": 1, "mxfp4": 2, "q4_k": 3, "q6_k": 4, "t5": 5}
F32, BF16 = 0, 1
MAX_TIERS = 8

_lib = None


class QmoeError(RuntimeError):
    pass


MAX_BATCH = 16


class GemvDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("R", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class Tier(ctypes.Structure):
    _fields_ = [("e_begin", ctypes.c_int32), ("e_end", ctypes.c_int32),
                ("fmt_gate_up", ctypes.c_int32), ("fmt_down", ctypes.c_int32),
                ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p),
                ("down", ctypes.c_void_p)]


_VP, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIGNATURES = {
    "qmoe_abi_version": (_I, []),
    "qmoe_status_string": (ctypes.c_char_p, [_I]),
    "qmoe_last_error": (ctypes.c_char_p, []),
    "qmoe_block_size": (_I, [_I]),
    "qmoe_tensor_bytes": (_SZ, [_I, _I, _I]),
    "qmoe_plane_offsets": (_I, [_I, _I, _I, ctypes.POINTER(_SZ)]),
    "qmoe_device_cu_count": (_I, []),
    "moe_route_workspace_size": (_SZ, [_I, _I, _I]),
    "moe_route": (_I, [_VP, _I, _I, _I, _VP, _VP, _I, _I, _I, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "moe_permute": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP, _VP]),
    "moe_route_decode_workspace_size": (_SZ, [_I, _I, _I]),
    "moe_route_decode": (_I, [_VP, _I, _I, _I, _VP, _VP, _I, _I, _I, _VP, _VP, _VP, _VP, _VP,
                              _VP, _VP, _SZ, _VP]),
    "moe_route_decode_noalloc_max_bytes": (_SZ, []),
    "moe_route_decode_noalloc": (_I, [_VP, _I, _I, _I, _VP, _VP, _I, _I, _I, _VP, _VP, _VP, _VP,
                                      _VP, _VP, _VP]),
    "moe_ffn_workspace_size": (_SZ, [_I, _I, _I]),
    "moe_ffn_tiered": (_I, [ctypes.POINTER(Tier), _I, _I, _I, _I, _VP, _I, _I, _I, _VP, _VP,
                            _VP, _VP, _SZ, _VP]),
    "qgemm_grouped_prefill_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "qgemm_grouped_prefill": (_I, [ctypes.POINTER(Tier), _I, _I, _I, _I, _VP, _I, _I, _I, _VP,
                                   _VP, _VP, _VP, _SZ, _VP]),
    "qgemm_grouped_prefill_mx": (_I, [ctypes.POINTER(Tier), _I, _I, _I, _I, _VP, _I, _I, _I, _VP,
                                      _VP, _VP, _VP, _SZ, _VP]),
    "moe_combine": (_I, [_VP, _VP, _VP, _I, _I, _I, _VP, _VP, _VP]),
    "qquantize_act_mxfp8": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP]),
    "qquantize_act_q8": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP]),
    "qgemv_q8_0_i8": (_I, [_VP, _I, _I, _VP, _VP, _I, _VP, _VP]),
    "qgemm_mxfp4_mxfp8": (_I, [_VP, _I, _I, _VP, _VP, _I, _VP, _VP]),
    "qgemm_q8_0_i8": (_I, [_VP, _I, _I, _VP, _VP, _I, _VP, _VP]),
    "qquantize_act_mxfp4": (_I, [_VP, _I, _I, _I, _VP, _VP, _VP]),
    "qdequant_act_mxfp4": (_I, [_VP, _VP, _I, _I, _VP, _I, _VP]),
    "qgemm_mxfp4_mxfp4": (_I, [_VP, _I, _I, _VP, _VP, _I, _VP, _I, _VP]),
    "moe_layer_decode_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moe_layer_decode": (_I, [ctypes.POINTER(Tier), _I, _I, _I, _I, _VP, _I, _I, _VP, _VP, _I,
                              _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "qmoe_stream_read": (_I, [_VP, _SZ, _I, _VP, _VP]),
    "qmoe_wave_latency": (_I, [_VP, _VP]),
    "qmoe_profile_enable": (_I, [_I]),
    "qmoe_profile_reset": (_I, []),
    "qmoe_profile_only": (_I, [ctypes.c_char_p]),
    "qmoe_profile_read": (_I, [ctypes.c_char_p, ctypes.POINTER(_I),
                               ctypes.POINTER(ctypes.c_double)]),
}
for _f in FORMATS:
    _SIGNATURES[f"qquantize_{_f}"] = (_I, [_VP, _I, _I, _VP, _VP])
    _SIGNATURES[f"qdequant_{_f}"] = (_I, [_VP, _I, _I, _VP, _VP])
    _SIGNATURES[f"qgemv_{_f}"] = (_I, [_VP, _I, _I, _VP, _I, _I, _VP, _VP])
_NORM_ARGS = [_VP, _I, _VP, _VP, _I, _VP, ctypes.c_double, _I, _I]
_SIGNATURES["qnorm"] = (_I, _NORM_ARGS + [_VP, _I, _VP])
for _f in ("q8", "mxfp8", "mxfp4"):
    _SIGNATURES[f"qnorm_act_{_f}"] = (_I, _NORM_ARGS + [_VP, _VP, _VP])
    _SIGNATURES[f"qswiglu_act_{_f}"] = (_I, [_VP, _VP, _I, ctypes.c_longlong, _I, _I, _VP, _VP,
                                             _VP])
_NORM_BLOCK_ARGS = [_VP, _I, _VP, ctypes.c_double, _VP, _I, _I, ctypes.c_double, _VP, _VP, _I,
                    ctypes.c_double, _VP, ctypes.c_double, _I, _I]
_SIGNATURES["qnorm_block"] = (_I, _NORM_BLOCK_ARGS + [_VP, _I, _VP])
for _f in ("q8", "mxfp8", "mxfp4"):
    _SIGNATURES[f"qnorm_block_act_{_f}"] = (_I, _NORM_BLOCK_ARGS + [_VP, _VP, _VP])
    _SIGNATURES[f"qlinear_{_f}"] = (_I, [_VP, _I, _I, _VP, _VP, _I, _VP, _I, _VP, _I, _VP, _I,
                                         _VP])
    _SIGNATURES[f"qglu_{_f}"] = (_I, [_VP, _VP, _I, _I, _VP, _VP, _I, _VP, _VP, _I, _VP, _I, _VP])
    _SIGNATURES[f"qglu_{_f}_act"] = (_I, [_VP, _VP, _I, _I, _VP, _VP, _I, _VP, _VP, _I, _VP, _VP,
                                          _VP])
_SIGNATURES["qgemv_batch"] = (_I, [_VP, _I, _VP])


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise QmoeError(f"{LIB_PATH} is missing: build it with "
                            "`python -m decode_moe_mul_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status, what):
    if status != 0:
        L = lib()
        raise QmoeError(f"{what}: {L.qmoe_status_string(status).decode()} "
                        f"({L.qmoe_last_error().decode()})")


def _torch():
    import torch
    return torch


def _stream():
    return ctypes.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(x):
    torch = _torch()
    if x.dtype == torch.float32:
        return F32
    if x.dtype == torch.bfloat16:
        return BF16
    raise QmoeError(f"activations must be float32 or bfloat16, got {x.dtype}")


def _need(cond, msg):
    if not cond:
        raise QmoeError(msg)


def _cuda_contig(*ts):
    for t in ts:
        if t is not None:
            _need(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")


def _alloc_bytes(n, device):
    """uint8 device buffer of >= n bytes with a 256-byte aligned start."""
    torch = _torch()
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ meta --

def abi_version():
    return lib().qmoe_abi_version()


def tensor_bytes(fmt, N, K):
    n = lib().qmoe_tensor_bytes(FORMATS[fmt], N, K)
    _need(n > 0 or N == 0, f"{fmt}: K={K} is not a multiple of the block")
    return n


def plane_offsets(fmt, N, K):
    offs = (ctypes.c_size_t * 4)()
    n = lib().qmoe_plane_offsets(FORMATS[fmt], N, K, offs)
    _check(0 if n > 0 else n, "qmoe_plane_offsets")
    return list(offs[:n])


def cu_count():
    return lib().qmoe_device_cu_count()


# --------------------------------------------------------------- formats --

def quantize(fmt, w, out=None):
    """fp32 [N, K] CUDA tensor -> packed uint8 tensor (plane layout)."""
    torch = _torch()
    _need(w.dtype == torch.float32 and w.dim() == 2, "w must be a float32 [N, K] tensor")
    _cuda_contig(w)
    N, K = w.shape
    if out is None:
        out = torch.zeros(tensor_bytes(fmt, N, K), dtype=torch.uint8, device=w.device)
    _check(getattr(lib(), f"qquantize_{fmt}")(_p(w), N, K, _p(out), _stream()), f"qquantize_{fmt}")
    return out


def dequantize(fmt, W, N, K, out=None):
    torch = _torch()
    _cuda_contig(W)
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32, device=W.device)
    _check(getattr(lib(), f"qdequant_{fmt}")(_p(W), N, K, _p(out), _stream()), f"qdequant_{fmt}")
    return out


def gemv_batch(items):
    """One launch for several independent GEMVs.  items: (fmt, W, N, K, x, out)
    tuples as gemv takes them (out required, [R, N] fp32); returns the outs."""
    torch = _torch()
    if len(items) > MAX_BATCH:
        raise ValueError(f"at most {MAX_BATCH} matrices per batch")
    descs = (GemvDesc * max(len(items), 1))()
    keep = []
    for i, (fmt, W, N, K, x, out) in enumerate(items):
        x2 = x if x.dim() == 2 else x.reshape(1, -1)
        _cuda_contig(W, x2, out)
        _need(x2.shape[1] == K, "x has the wrong length")
        _need(tuple(out.shape) == (x2.shape[0], N) and out.dtype == torch.float32,
              "out must be fp32 [R, N]")
        keep.append(x2)
        descs[i] = GemvDesc(FORMATS[fmt], N, K, _dtype_code(x2), x2.shape[0], 0,
                            _p(W), _p(x2), _p(out))
    _check(lib().qgemv_batch(descs, len(items), _stream()), "qgemv_batch")
    return [it[5] for it in items]


def gemv(fmt, W, N, K, x, out=None):
    """y [R, N] = x [R, K] . deq(W)^T."""
    torch = _torch()
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    _cuda_contig(W, x2)
    _need(x2.shape[1] == K, "x has the wrong length")
    R = x2.shape[0]
    if out is None:
        out = torch.empty((R, N), dtype=torch.float32, device=x.device)
    _check(getattr(lib(), f"qgemv_{fmt}")(_p(W), N, K, _p(x2), _dtype_code(x2), R, _p(out),
                                          _stream()), f"qgemv_{fmt}")
    return out


# --------------------------------------------------------------- routing --

def route_workspace(T, H, E, device="cuda"):
    return _alloc_bytes(lib().moe_route_workspace_size(T, H, E), device)


def route(x, Wr, bias, k, n_shared=0, logits=False, ws=None):
    """ids [T, k+n_shared] int32, p [T, k+n_shared] fp32 (and logits [T, E])."""
    torch = _torch()
    _cuda_contig(x, Wr, bias)
    T, H = x.shape
    E = Wr.shape[0]
    kt = k + n_shared
    ids = torch.empty((T, kt), dtype=torch.int32, device=x.device)
    p = torch.empty((T, kt), dtype=torch.float32, device=x.device)
    lg = torch.empty((T, E), dtype=torch.float32, device=x.device) if logits else None
    if ws is None:
        ws = route_workspace(T, H, E, x.device)
    _check(lib().moe_route(_p(x), _dtype_code(x), T, H, _p(Wr), _p(bias), E, k, n_shared,
                           _p(ids), _p(p), _p(lg), _p(ws), ws.numel(), _stream()), "moe_route")
    return (ids, p, lg) if logits else (ids, p)


def route_decode_workspace(T, H, E, device="cuda"):
    """Workspace of moe_route_decode: zero-filled, as its counters require."""
    torch = _torch()
    n = lib().moe_route_decode_workspace_size(T, H, E)
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


def route_decode(x, Wr, bias, k, n_shared=0, logits=False, ws=None):
    """moe_route + moe_permute in one launch (T <= 16):
    ids, p, offsets, perm, inv_perm (and logits [T, E])."""
    torch = _torch()
    _cuda_contig(x, Wr, bias)
    T, H = x.shape
    E = Wr.shape[0]
    kt = k + n_shared
    dev = x.device
    ids = torch.empty((T, kt), dtype=torch.int32, device=dev)
    p = torch.empty((T, kt), dtype=torch.float32, device=dev)
    lg = torch.empty((T, E), dtype=torch.float32, device=dev) if logits else None
    offsets = torch.empty(E + n_shared + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(T * kt, 1), dtype=torch.int32, device=dev)
    inv = torch.empty(max(T * kt, 1), dtype=torch.int32, device=dev)
    if ws is None:
        ws = route_decode_workspace(T, H, E, dev)
    _check(lib().moe_route_decode(_p(x), _dtype_code(x), T, H, _p(Wr), _p(bias), E, k, n_shared,
                                  _p(ids), _p(p), _p(lg), _p(offsets), _p(perm), _p(inv),
                                  _p(ws), ws.numel(), _stream()), "moe_route_decode")
    out = (ids, p, offsets, perm, inv)
    return out + (lg,) if logits else out


def route_decode_noalloc(x, Wr, bias, k, n_shared=0, logits=False, out=None):
    """moe_route_decode_noalloc: as route_decode, with the library's own
    device scratch instead of a workspace (the call allocates nothing; the
    output tensors are allocated here unless `out` = (ids, p, offsets, perm,
    inv_perm[, logits]) is given)."""
    torch = _torch()
    _cuda_contig(x, Wr, bias)
    T, H = x.shape
    E = Wr.shape[0]
    kt = k + n_shared
    dev = x.device
    if out is None:
        out = (torch.empty((T, kt), dtype=torch.int32, device=dev),
               torch.empty((T, kt), dtype=torch.float32, device=dev),
               torch.empty(E + n_shared + 1, dtype=torch.int32, device=dev),
               torch.empty(max(T * kt, 1), dtype=torch.int32, device=dev),
               torch.empty(max(T * kt, 1), dtype=torch.int32, device=dev))
        if logits:
            out = out + (torch.empty((T, E), dtype=torch.float32, device=dev),)
    ids, p, offsets, perm, inv = out[:5]
    lg = out[5] if len(out) > 5 else None
    _check(lib().moe_route_decode_noalloc(_p(x), _dtype_code(x), T, H, _p(Wr), _p(bias), E, k,
                                          n_shared, _p(ids), _p(p), _p(lg), _p(offsets),
                                          _p(perm), _p(inv), _stream()),
           "moe_route_decode_noalloc")
    return out


def permute(ids, E, out=None):
    """offsets [E+1], perm [A], inv_perm [A] (int32) of ids [T, k]."""
    torch = _torch()
    _cuda_contig(ids)
    _need(ids.dtype == torch.int32, "ids must be int32")
    T, k = ids.shape if ids.dim() == 2 else (ids.numel(), 1)
    A = T * k
    if out is None:
        out = (torch.empty(E + 1, dtype=torch.int32, device=ids.device),
               torch.empty(max(A, 1), dtype=torch.int32, device=ids.device),
               torch.empty(max(A, 1), dtype=torch.int32, device=ids.device))
    offsets, perm, inv = out
    _check(lib().moe_permute(_p(ids), T, k, E, _p(offsets), _p(perm), _p(inv), _stream()),
           "moe_permute")
    return offsets, perm[:A], inv[:A]


# ------------------------------------------------------------ expert FFN --

def tiers_struct(tiers):
    """tiers: iterable of (e_begin, e_end, fmt_gate_up, fmt_down, gate, up,
    down) with packed uint8 CUDA tensors -> ctypes array (keep tensors alive)."""
    tiers = list(tiers)
    arr = (Tier * len(tiers))()
    for i, (b, e, fgu, fd, g, u, d) in enumerate(tiers):
        _cuda_contig(g, u, d)
        arr[i] = Tier(b, e, FORMATS[fgu], FORMATS[fd], g.data_ptr(), u.data_ptr(), d.data_ptr())
    return arr


def ffn_workspace(T, k, F, device="cuda"):
    return _alloc_bytes(lib().moe_ffn_workspace_size(T, k, F), device)


def prefill_workspace(T, k, E, H, F, device="cuda"):
    return _alloc_bytes(lib().qgemm_grouped_prefill_workspace_size(T, k, E, H, F), device)


def _ffn_call(name, tiers, E, H, F, x, k, offsets, perm, out, ws):
    torch = _torch()
    _cuda_contig(x, offsets, perm)
    T = x.shape[0]
    arr = tiers if isinstance(tiers, ctypes.Array) else tiers_struct(tiers)
    if out is None:
        out = torch.empty((max(T * k, 1), H), dtype=torch.float32, device=x.device)
    fn = getattr(lib(), name)
    _check(fn(arr, len(arr), E, H, F, _p(x), _dtype_code(x), T, k, _p(offsets), _p(perm),
              _p(out), _p(ws), 0 if ws is None else ws.numel(), _stream()), name)
    return out


def ffn_tiered(tiers, E, H, F, x, k, offsets, perm, out=None, ws=None):
    """o [T*k, H] in permuted order (decode kernels)."""
    if ws is None:
        ws = ffn_workspace(x.shape[0], k, F, x.device)
    return _ffn_call("moe_ffn_tiered", tiers, E, H, F, x, k, offsets, perm, out, ws)


def grouped_prefill(tiers, E, H, F, x, k, offsets, perm, out=None, ws=None):
    """o [T*k, H] in permuted order (matrix-core grouped GEMM)."""
    if ws is None:
        ws = prefill_workspace(x.shape[0], k, E, H, F, x.device)
    return _ffn_call("qgemm_grouped_prefill", tiers, E, H, F, x, k, offsets, perm, out, ws)


def grouped_prefill_mx(tiers, E, H, F, x, k, offsets, perm, out=None, ws=None):
    """As grouped_prefill, with MXFP4/MXFP4 tiers on the block-scaled matrix
    cores against MXFP8 activations."""
    if ws is None:
        ws = prefill_workspace(x.shape[0], k, E, H, F, x.device)
    return _ffn_call("qgemm_grouped_prefill_mx", tiers, E, H, F, x, k, offsets, perm, out, ws)


def combine(o, inv_perm, p, T, k, H, shared=None, out=None):
    torch = _torch()
    _cuda_contig(o, inv_perm, p, shared)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=o.device)
    _check(lib().moe_combine(_p(o), _p(inv_perm), _p(p), T, k, H, _p(shared), _p(out),
                             _stream()), "moe_combine")
    return out


def quantize_act_mxfp8(x):
    """Activations [R, K] (float32 or bfloat16) -> MXFP8 codes [R, K] uint8
    (E4M3) and scales [R, K/32] uint8 (E8M0)."""
    torch = _torch()
    _cuda_contig(x)
    R, K = x.shape
    codes = torch.empty((R, K), dtype=torch.uint8, device=x.device)
    scales = torch.empty((R, max(K // 32, 1)), dtype=torch.uint8, device=x.device)
    _check(lib().qquantize_act_mxfp8(_p(x), _dtype_code(x), R, K, _p(codes), _p(scales),
                                     _stream()), "qquantize_act_mxfp8")
    return codes, scales


def quantize_act_q8(x):
    """Activations [R, K] (float32 or bfloat16) -> int8 codes [R, K] and fp32
    block scales [R, K/32]."""
    torch = _torch()
    _cuda_contig(x)
    R, K = x.shape
    q = torch.empty((R, K), dtype=torch.int8, device=x.device)
    d = torch.empty((R, max(K // 32, 1)), dtype=torch.float32, device=x.device)
    _check(lib().qquantize_act_q8(_p(x), _dtype_code(x), R, K, _p(q), _p(d), _stream()),
           "qquantize_act_q8")
    return q, d


def gemv_q8_0_i8(W, N, K, q, d, out=None):
    """y [R, N] = Q8_0 W [N, K] times the int8 activations (q, d)."""
    torch = _torch()
    _cuda_contig(W, q, d)
    R = q.shape[0]
    if out is None:
        out = torch.empty((R, N), dtype=torch.float32, device=q.device)
    _check(lib().qgemv_q8_0_i8(_p(W), N, K, _p(q), _p(d), R, _p(out), _stream()),
           "qgemv_q8_0_i8")
    return out


def gemm_q8_0_i8(W, N, K, q, d, out=None):
    """y [R, N] = Q8_0 W [N, K] times the int8 activations (q, d) on the
    int8 matrix cores (prefill-sized R)."""
    torch = _torch()
    _cuda_contig(W, q, d)
    R = q.shape[0]
    if out is None:
        out = torch.empty((R, N), dtype=torch.float32, device=q.device)
    _check(lib().qgemm_q8_0_i8(_p(W), N, K, _p(q), _p(d), R, _p(out), _stream()),
           "qgemm_q8_0_i8")
    return out


def gemm_mxfp4_mxfp8(W, N, K, codes, scales, out=None):
    """y [R, N] = W (MXFP4 [N, K]) times the MXFP8 activations."""
    torch = _torch()
    _cuda_contig(W, codes, scales)
    R = codes.shape[0]
    if out is None:
        out = torch.empty((R, N), dtype=torch.float32, device=codes.device)
    _check(lib().qgemm_mxfp4_mxfp8(_p(W), N, K, _p(codes), _p(scales), R, _p(out), _stream()),
           "qgemm_mxfp4_mxfp8")
    return out


# ---------------------------------------------------- 4-bit activations --

# These calls take a few microseconds on the GPU for a decode row, and so do a
# launch and each tensor that torch allocates.  Their own host side is kept
# short: one condition over everything a call needs (what is wrong is worked out
# only when something is), pointers as plain ints, the raw stream handle.

ACT_FORMATS = ("q8", "mxfp8", "mxfp4")
_th = None           # torch, once a call has needed it, and two of its functions
_device = _stream_of = None
_FLOAT = {}          # output and activation types -> dtype codes
_ACT_TYPES = {}      # format -> (values per code, code type, scale type)
_MOST = 2 ** 31 - 1  # sizes pass as C ints, of which ctypes keeps the low bits silently


def _load_torch():
    global _th, _device, _stream_of
    torch = _torch()
    _device, _stream_of = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _FLOAT.update({torch.float32: F32, torch.bfloat16: BF16})
    _ACT_TYPES.update({"q8": (1, torch.int8, torch.float32),
                       "mxfp8": (1, torch.uint8, torch.uint8),
                       "mxfp4": (2, torch.uint8, torch.uint8)})
    _th = torch
    return torch


def _launch(name, index, *args):
    """Call entry point `name` with GPU `index` current, on that GPU's current
    stream."""
    fn = getattr(_lib or lib(), name)
    if index == _device():
        st = fn(*args, _stream_of(index))
    else:
        with _th.cuda.device(index):
            st = fn(*args, _stream_of(index))
    if st:
        _check(st, name)


def _is(t, shape, dtype, index):
    return (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous())


def _refuse(what, t, shape, dtype, index):
    """Raise for a tensor that _is not what it has to be."""
    place = f"GPU {index}" if index >= 0 else "a GPU"
    raise QmoeError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                    f"{place}, not {t.dtype} {tuple(t.shape)} on {t.device}"
                    f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def _rows(x, what):
    """(R, K, GPU index, dtype code) of activations [R, K]."""
    code, index = _FLOAT.get(x.dtype), x.get_device()
    if code is None or index < 0 or x.dim() != 2 or not x.is_contiguous():
        raise QmoeError(f"{what} must be a contiguous float32 or bfloat16 CUDA tensor [R, K], "
                        f"not {x.dtype} {tuple(x.shape)} on {x.device}")
    R, K = x.shape
    if R > _MOST or K > _MOST:
        raise QmoeError(f"{what} [{R}, {K}]: sizes are below 2^31")
    return R, K, index, code


def _float_out(out, dtype, like, shape, index):
    """(out, dtype code): a new tensor unless out is given."""
    if out is None:
        dtype = _th.float32 if dtype is None else dtype
    elif not _is(out, shape, out.dtype if dtype is None else dtype, index):
        _refuse("out", out, shape, dtype or out.dtype, index)
    else:
        dtype = out.dtype
    code = _FLOAT.get(dtype)
    if code is None:
        raise QmoeError(f"outputs are float32 or bfloat16, not {dtype}")
    return (like.new_empty(shape, dtype=dtype) if out is None else out), code


def _act_out(fmt, like, R, K, index, out):
    """(codes, scales) of activation format `fmt` for [R, K]."""
    kinds = _ACT_TYPES.get(fmt)
    if kinds is None:
        raise QmoeError(f"activation format {fmt!r} is not one of {ACT_FORMATS}")
    if K <= 0 or K % 32:
        raise QmoeError(f"K={K} is not a multiple of 32")
    per, ct, st = kinds
    if out is None:
        return like.new_empty((R, K // per), dtype=ct), like.new_empty((R, K // 32), dtype=st)
    codes, scales = out
    if not _is(codes, (R, K // per), ct, index):
        _refuse("codes", codes, (R, K // per), ct, index)
    if not _is(scales, (R, K // 32), st, index):
        _refuse("scales", scales, (R, K // 32), st, index)
    return codes, scales


def _act_in(codes, scales, K):
    """(R, GPU index) of MXFP4 activations [R, K]."""
    u8, index, R = _th.uint8, codes.get_device(), codes.shape[0] if codes.dim() else 0
    if index < 0 or not _is(codes, (R, K // 2), u8, index):
        _refuse("codes", codes, (R, K // 2), u8, index)
    if not _is(scales, (R, K // 32), u8, index):
        _refuse("scales", scales, (R, K // 32), u8, index)
    if R > _MOST or K > _MOST:
        raise QmoeError(f"activations [{R}, {K}]: sizes are below 2^31")
    return R, index


def quantize_act_mxfp4(x, out=None):
    """Activations [R, K] (float32 or bfloat16) -> MXFP4 codes [R, K/2] uint8
    (two E2M1 codes per byte, low nibble first) and scales [R, K/32] uint8
    (E8M0)."""
    _th or _load_torch()
    R, K, index, xd = _rows(x, "x")
    codes, scales = _act_out("mxfp4", x, R, K, index, out)
    _launch("qquantize_act_mxfp4", index, x.data_ptr(), xd, R, K, codes.data_ptr(),
            scales.data_ptr())
    return codes, scales


def dequantize_act_mxfp4(codes, scales, dtype=None, out=None):
    """The values [R, K] of MXFP4 activations (float32 unless dtype says
    bfloat16)."""
    _th or _load_torch()
    K = 2 * codes.shape[-1] if codes.dim() else 0
    R, index = _act_in(codes, scales, K)
    out, yd = _float_out(out, dtype, codes, (R, K), index)
    _launch("qdequant_act_mxfp4", index, codes.data_ptr(), scales.data_ptr(), R, K,
            out.data_ptr(), yd)
    return out


def _norm_args(x, w, eps, res, res_out):
    R, K, index, xd = _rows(x, "x")
    f32 = _th.float32
    if not _is(w, (K,), f32, index):
        _refuse("w", w, (K,), f32, index)
    if res is None:
        if res_out is not None:
            raise QmoeError("res_out without res")
        return index, R, K, None, (x.data_ptr(), xd, None, None, 0, w.data_ptr(), eps, R, K)
    rd, shape = _FLOAT.get(res.dtype), x.shape
    if rd is None or not _is(res, shape, res.dtype, index):
        _refuse("res", res, shape, "float32 or bfloat16", index)
    at = res.data_ptr()
    if res_out is None:
        res_out = _th.empty_like(res)
    elif res_out is not res and not _is(res_out, shape, res.dtype, index):
        _refuse("res_out", res_out, shape, res.dtype, index)
    return index, R, K, res_out, (x.data_ptr(), xd, at, res_out.data_ptr(), rd, w.data_ptr(),
                                  eps, R, K)


def norm(x, w, eps, res=None, res_out=None, dtype=None, out=None):
    """RMS norm of the rows of x [R, K], or of h = x + res: y = h * w /
    sqrt(mean(h^2) + eps) in float32, or dtype.  Returns y, with res (y, h);
    h has res' type and goes to res_out (a new tensor unless given; res itself
    for an update in place)."""
    _th or _load_torch()
    index, R, K, h, args = _norm_args(x, w, eps, res, res_out)
    out, yd = _float_out(out, dtype, x, (R, K), index)
    _launch("qnorm", index, *args, out.data_ptr(), yd)
    return out if res is None else (out, h)


def norm_act(fmt, x, w, eps, res=None, res_out=None, out=None):
    """norm's float32 rows in activation format fmt ("q8", "mxfp8", "mxfp4"):
    (codes, scales), with res (codes, scales, h)."""
    _th or _load_torch()
    index, R, K, h, args = _norm_args(x, w, eps, res, res_out)
    codes, scales = _act_out(fmt, x, R, K, index, out)
    _launch("qnorm_act_" + fmt, index, *args, codes.data_ptr(), scales.data_ptr())
    return (codes, scales) if res is None else (codes, scales, h)


def swiglu_act(fmt, gate, up, out=None):
    """gate / (1 + exp(-gate)) * up [R, K] in activation format fmt: (codes,
    scales).  gate and up are float32 or bfloat16, with contiguous rows; the
    rows may lie further apart (the two halves of one [R, 2K] tensor)."""
    _th or _load_torch()
    xd, index, shape = _FLOAT.get(gate.dtype), gate.get_device(), gate.shape
    if (xd is None or index < 0 or len(shape) != 2 or up.shape != shape
            or up.dtype is not gate.dtype or up.get_device() != index):
        raise QmoeError("gate and up must be float32 or bfloat16 CUDA tensors [R, K] of one "
                        "type on one GPU")
    R, K = shape
    if R > _MOST or K > _MOST:
        raise QmoeError(f"gate and up [{R}, {K}]: sizes are below 2^31")
    ld = K
    if R > 0:
        (ld, one), (ld_up, one_up) = gate.stride(), up.stride()
        if R == 1:
            ld = ld_up = K   # the distance of a single row says nothing
        if one != 1 or one_up != 1 or ld != ld_up:
            raise QmoeError("gate and up must have contiguous rows, equally far apart")
    codes, scales = _act_out(fmt, gate, R, K, index, out)
    _launch("qswiglu_act_" + fmt, index, gate.data_ptr(), up.data_ptr(), xd, ld, R, K,
            codes.data_ptr(), scales.data_ptr())
    return codes, scales


def gemm_mxfp4_mxfp4(W, N, K, codes, scales, dtype=None, out=None):
    """y [R, N] (float32 unless dtype says bfloat16) = W (MXFP4 [N, K]) times
    the MXFP4 activations; R from one decode row to a prefill chunk."""
    _th or _load_torch()
    R, index = _act_in(codes, scales, K)
    if N > _MOST:
        raise QmoeError(f"W [{N}, {K}]: sizes are below 2^31")
    if (N < 0 or W.dtype is not codes.dtype or W.get_device() != index or not W.is_contiguous()
            or W.numel() < -(-N * K // 512) * 256 + -(-N * K // 8192) * 256):
        raise QmoeError("W must be a packed MXFP4 [N, K] tensor on the activations' GPU")
    out, yd = _float_out(out, dtype, codes, (R, N), index)
    _launch("qgemm_mxfp4_mxfp4", index, W.data_ptr(), N, K, codes.data_ptr(), scales.data_ptr(),
            R, out.data_ptr(), yd)
    return out


# -------------------------------------- the dense block, fused products --

ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4, "relu2": 5}


def _product_refused(fmt, N, K, codes, scales, act):
    """Raise for what is wrong with a product's operands."""
    kinds = _ACT_TYPES.get(fmt)
    if kinds is None:
        raise QmoeError(f"activation format {fmt!r} is not one of {ACT_FORMATS}")
    if act not in ACTIVATIONS:
        raise QmoeError(f"activation {act!r} is not one of {tuple(ACTIVATIONS)}")
    if K <= 0 or K % 32 or K > _MOST or not 0 <= N <= _MOST:
        raise QmoeError(f"W [{N}, {K}]: N is at least 0, K a multiple of 32, both below 2^31")
    per, ct, st = kinds
    index, R = codes.get_device(), codes.shape[0] if codes.dim() else 0
    if index < 0 or not _is(codes, (R, K // per), ct, index):
        _refuse("codes", codes, (R, K // per), ct, index)
    if not _is(scales, (R, K // 32), st, index):
        _refuse("scales", scales, (R, K // 32), st, index)
    if R > _MOST:
        raise QmoeError(f"activations [{R}, {K}]: sizes are below 2^31")
    raise QmoeError(f"weights must be packed {'Q8_0' if fmt == 'q8' else 'MXFP4'} [{N}, {K}] "
                    "tensors on the activations' GPU")


def _product_args(fmt, N, K, codes, scales, act, W, W2=None):
    """(R, GPU index, activation code) of a product's operands."""
    kinds, code = _ACT_TYPES.get(fmt), ACTIVATIONS.get(act)
    index, shape = codes.get_device(), codes.shape
    if kinds is not None and code is not None and index >= 0 and len(shape) == 2:
        per, ct, st = kinds
        R, u8 = shape[0], _th.uint8
        # two planes, each from a 256-byte boundary on: int8 codes and fp16 scales, or
        # 4-bit codes and one byte a scale
        need = ((N * K + 255 >> 8) + (N * K + 4095 >> 12) if per == 1 and ct is not u8 else
                (N * K + 511 >> 9) + (N * K + 8191 >> 13)) << 8
        if (0 < K <= _MOST and K % 32 == 0 and 0 <= N <= _MOST and R <= _MOST
                and shape[1] == K // per and codes.dtype is ct and codes.is_contiguous()
                and scales.dtype is st and scales.shape == (R, K // 32)
                and scales.get_device() == index and scales.is_contiguous()
                and W.dtype is u8 and W.get_device() == index and W.is_contiguous()
                and W.numel() >= need
                and (W2 is None or W2.dtype is u8 and W2.get_device() == index
                     and W2.is_contiguous() and W2.numel() >= need)):
            return R, index, code
    _product_refused(fmt, N, K, codes, scales, act)


def _bias(b, N, index, what):
    if b is None:
        return None
    if not _is(b, (N,), _th.float32, index):
        _refuse(what, b, (N,), _th.float32, index)
    return b.data_ptr()


def linear(fmt, W, N, K, codes, scales, bias=None, act=None, res=None, dtype=None, out=None):
    """y [R, N] = act(x W^T + bias) + res (float32 unless dtype says bfloat16) of
    activations x in format fmt ("q8", "mxfp8", "mxfp4": codes, scales) and packed
    weights W [N, K], Q8_0 for "q8" and MXFP4 for the others; R from one decode
    row to a prefill chunk.  bias: float32 [N]; act: one of ACTIVATIONS; res:
    float32 or bfloat16 [R, N].  out may be res itself: the residual stream
    updated in place."""
    _th or _load_torch()
    R, index, code = _product_args(fmt, N, K, codes, scales, act, W)
    bias = _bias(bias, N, index, "bias")
    rd, at = 0, None
    if res is not None:
        rd, at = _FLOAT.get(res.dtype), res.data_ptr()
        if rd is None or not _is(res, (R, N), res.dtype, index):
            _refuse("res", res, (R, N), "float32 or bfloat16", index)
    out, yd = _float_out(out, dtype, codes, (R, N), index)
    _launch("qlinear_" + fmt, index, W.data_ptr(), N, K, codes.data_ptr(), scales.data_ptr(), R,
            bias, code, at, rd, out.data_ptr(), yd)
    return out


def glu(fmt, Wg, Wu, N, K, codes, scales, act="silu", bias_gate=None, bias_up=None, dtype=None,
        out=None):
    """y [R, N] = act(x Wg^T + bias_gate) * (x Wu^T + bias_up), operands as linear
    takes them, in float32 unless dtype says bfloat16."""
    _th or _load_torch()
    R, index, code = _product_args(fmt, N, K, codes, scales, act, Wg, Wu)
    bg, bu = _bias(bias_gate, N, index, "bias_gate"), _bias(bias_up, N, index, "bias_up")
    out, yd = _float_out(out, dtype, codes, (R, N), index)
    _launch("qglu_" + fmt, index, Wg.data_ptr(), Wu.data_ptr(), N, K, codes.data_ptr(),
            scales.data_ptr(), R, bg, bu, code, out.data_ptr(), yd)
    return out


def glu_act(fmt, Wg, Wu, N, K, codes, scales, act="silu", bias_gate=None, bias_up=None, out=None):
    """glu's float32 rows as activations (codes, scales) of the next product, in
    the same format fmt (the sums may be in another order than glu's)."""
    _th or _load_torch()
    R, index, code = _product_args(fmt, N, K, codes, scales, act, Wg, Wu)
    bg, bu = _bias(bias_gate, N, index, "bias_gate"), _bias(bias_up, N, index, "bias_up")
    oc, os_ = _act_out(fmt, codes, R, N, index, out)
    _launch("qglu_" + fmt + "_act", index, Wg.data_ptr(), Wu.data_ptr(), N, K, codes.data_ptr(),
            scales.data_ptr(), R, bg, bu, code, oc.data_ptr(), os_.data_ptr())
    return oc, os_


def _norm_block_args(x, res, w, eps, w_post, eps_post, gate, scale, res_scale, res_out):
    R, K, index, xd = _rows(x, "x")
    f32 = _th.float32
    if not _is(w, (K,), f32, index):
        _refuse("w", w, (K,), f32, index)
    post = None
    if w_post is not None:
        if not _is(w_post, (K,), f32, index):
            _refuse("w_post", w_post, (K,), f32, index)
        post = w_post.data_ptr()
    rd, shape = _FLOAT.get(res.dtype), x.shape
    if rd is None or not _is(res, shape, res.dtype, index):
        _refuse("res", res, shape, "float32 or bfloat16", index)
    if res_out is None:
        res_out = _th.empty_like(res)
    elif res_out is not res and not _is(res_out, shape, res.dtype, index):
        _refuse("res_out", res_out, shape, res.dtype, index)
    gd, gates, gp = 0, 1, None
    if gate is not None:
        gates = gate.shape[0] if gate.dim() == 2 else 1
        gd = _FLOAT.get(gate.dtype)
        want = (gates, K) if gate.dim() == 2 else (K,)
        if gd is None or not _is(gate, want, gate.dtype, index):
            _refuse("gate", gate, want, "float32 or bfloat16", index)
        gates = gates if R else 1
        if gates < 1 or R % gates:
            raise QmoeError(f"gate [{gates}, {K}]: its rows must divide x's {R}")
        gp = gate.data_ptr()
    return index, R, K, res_out, (
        x.data_ptr(), xd, post, eps if eps_post is None else eps_post, gp, gd, gates, scale,
        res.data_ptr(), res_out.data_ptr(), rd, res_scale, w.data_ptr(), eps, R, K)


def norm_block(x, res, w, eps, w_post=None, eps_post=None, gate=None, scale=1.0, res_scale=1.0,
               res_out=None, dtype=None, out=None):
    """The norms around a block: h = res_scale * res + scale * gate * z, where z is
    the RMS norm of the block's output x [R, K] with weights w_post (x itself
    without them), and y, the RMS norm of h with weights w.  eps_post is eps
    unless given.  gate: float32 or bfloat16, [K], or [G, K] for R / G rows each.
    Returns (y, h): y float32 unless dtype says bfloat16, h in res' type, to
    res_out (a new tensor unless given; res itself for an update in place)."""
    _th or _load_torch()
    index, R, K, h, args = _norm_block_args(x, res, w, eps, w_post, eps_post, gate, scale,
                                            res_scale, res_out)
    out, yd = _float_out(out, dtype, x, (R, K), index)
    _launch("qnorm_block", index, *args, out.data_ptr(), yd)
    return out, h


def norm_block_act(fmt, x, res, w, eps, w_post=None, eps_post=None, gate=None, scale=1.0,
                   res_scale=1.0, res_out=None, out=None):
    """norm_block's float32 y in activation format fmt ("q8", "mxfp8", "mxfp4"):
    (codes, scales, h)."""
    _th or _load_torch()
    index, R, K, h, args = _norm_block_args(x, res, w, eps, w_post, eps_post, gate, scale,
                                            res_scale, res_out)
    codes, scales = _act_out(fmt, x, R, K, index, out)
    _launch("qnorm_block_act_" + fmt, index, *args, codes.data_ptr(), scales.data_ptr())
    return codes, scales, h


def layer_decode_workspace(T, H, E, F, k, n_shared=0, device="cuda"):
    """Workspace of moe_layer_decode: zero-filled, as its barrier counter requires."""
    torch = _torch()
    n = lib().moe_layer_decode_workspace_size(T, H, E, F, k, n_shared)
    return torch.zeros(max(int(n), 1), dtype=torch.uint8, device=device)


def layer_decode_error(ws):
    """The error word of a moe_layer_decode workspace (waits for the stream):
    nonzero once a grid-barrier wait of some call on it ran out, which makes
    that call's outputs invalid.  The word stays set until cleared."""
    torch = _torch()
    torch.cuda.current_stream().synchronize()
    return int(ws[:4].view(torch.int32).item())


def check_layer_decode(ws):
    """Raise QmoeError if the workspace's error word is set (clearing it, so
    that the workspace can be used again)."""
    if layer_decode_error(ws):
        ws[:4].zero_()
        raise QmoeError("moe_layer_decode: a grid-barrier wait ran out; the outputs of the "
                        "calls since the workspace was last checked are invalid")


def layer_decode(tiers, E, H, F, x, Wr, bias, k, n_shared=0, out=None, ws=None, check=True):
    """The whole routed-expert layer for decode rows (T <= 16) in one launch:
    y [T, H] and the routing ids, p, offsets, perm, inv_perm.  check: wait
    for the call and raise if its barrier error word is set (callers that
    queue many calls may pass False and call check_layer_decode(ws) once
    afterwards: the word is sticky)."""
    torch = _torch()
    _cuda_contig(x, Wr, bias)
    T = x.shape[0]
    dev = x.device
    kt, E_total = k + n_shared, E + n_shared
    arr = tiers if isinstance(tiers, ctypes.Array) else tiers_struct(tiers)
    ids = torch.empty((T, kt), dtype=torch.int32, device=dev)
    p = torch.empty((T, kt), dtype=torch.float32, device=dev)
    offsets = torch.empty(E_total + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(T * kt, 1), dtype=torch.int32, device=dev)
    inv = torch.empty(max(T * kt, 1), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=dev)
    if ws is None:
        ws = layer_decode_workspace(T, H, E, F, k, n_shared, dev)
    _check(lib().moe_layer_decode(arr, len(arr), E, H, F, _p(x), _dtype_code(x), T, _p(Wr),
                                  _p(bias), k, n_shared, _p(ids), _p(p), _p(offsets), _p(perm),
                                  _p(inv), _p(out), _p(ws), ws.numel(), _stream()),
           "moe_layer_decode")
    if check:
        check_layer_decode(ws)
    return out, ids, p, offsets, perm, inv


# ------------------------------------------------------------ measurement --

def wave_latency():
    """qmoe_wave_latency: one wave's dependent-step latencies (shader cycles)
    and the routing top-k's cost, as a dict."""
    torch = _torch()
    out = torch.zeros(8, dtype=torch.int64, device="cuda")
    _check(lib().qmoe_wave_latency(_p(out), _stream()), "qmoe_wave_latency")
    v = out.cpu().tolist()
    return {"valu_dependent_cycles": v[0], "dpp_wave_max_cycles": v[1],
            "ballot_round_trip_cycles": v[2], "wave_topk_512_k10_cycles": v[3],
            "lane_sort_8_cycles": v[4], "shader_clock_mhz": v[5]}


def stream_read(buf, blocks_per_cu=8, sink=None):
    """One streaming read of the CUDA tensor buf (qmoe_stream_read)."""
    torch = _torch()
    _cuda_contig(buf)
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device=buf.device)
    nbytes = buf.numel() * buf.element_size()
    _check(lib().qmoe_stream_read(_p(buf), nbytes, blocks_per_cu, _p(sink), _stream()),
           "qmoe_stream_read")
    return sink


# -------------------------------------------------------------- profiling --

def profile_enable(on=True):
    _check(lib().qmoe_profile_enable(1 if on else 0), "qmoe_profile_enable")


def profile_only(name=None):
    """Record only launches of kernel `name` (None: all)."""
    _check(lib().qmoe_profile_only(None if name is None else name.encode()), "qmoe_profile_only")


def profile_reset():
    _check(lib().qmoe_profile_reset(), "qmoe_profile_reset")


def profile_read(name):
    n = ctypes.c_int(0)
    ms = ctypes.c_double(0.0)
    _check(lib().qmoe_profile_read(name.encode(), ctypes.byref(n), ctypes.byref(ms)),
           "qmoe_profile_read")
    return n.value, ms.value
