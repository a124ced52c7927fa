"""Entry points of a decoder's other layers: gated linear recurrence, q/k norm with
rotation, paged key-value cache and its decode attention.

The same thin binding as the rest of the package: tensors' pointers, sizes and strides go
into the C ABI (``include/gdr.h``), status codes come back as exceptions, all arithmetic
runs in the CUDA kernels. Inputs may be views (any batch, token and head stride, the last
dimension dense); outputs are dense.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import warnings
from typing import Optional

import torch

from .build import host_path
from . import (GDR_BF16, GDR_ERR_INVALID_ARG, GDR_F32, GDR_OK, LIB_PATH, GdrError, load_library)

SCAN_CHECKPOINT = 64        # GDR_SCAN_CHECKPOINT
_DTYPE = {torch.bfloat16: GDR_BF16, torch.float32: GDR_F32}
_i, _l, _p, _f, _z = (ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float,
                      ctypes.c_size_t)


class gdr_scan_dims(ctypes.Structure):
    _fields_ = [(n, _i) for n in ("B", "T", "D", "x_dtype", "g_dtype", "h_dtype",
                                  "gated_input")] + \
               [(n, _l) for n in ("x_stride_b", "x_stride_t", "g_stride_b", "g_stride_t",
                                  "dh_stride_b", "dh_stride_t")]


class gdr_qk_dims(ctypes.Structure):
    _fields_ = [(n, _i) for n in ("B", "T", "HQ", "HK", "D", "R", "in_dtype", "out_dtype",
                                  "interleaved", "position_bits", "table_rows")] + \
               [("eps", _f)] + \
               [(f"{n}_stride_{d}", _l) for n in "qkv" for d in "bth"]


class gdr_paged_cache(ctypes.Structure):
    _fields_ = [(n, _i) for n in ("num_pages", "page_size", "HK", "D", "dtype", "max_pages")] + \
               [(n, _l) for n in ("page_stride", "token_stride", "head_stride")]


class gdr_attn_dims(ctypes.Structure):
    _fields_ = [(n, _i) for n in ("B", "HQ", "q_dtype", "out_dtype", "window")] + \
               [("scale", _f), ("q_stride_b", _l), ("q_stride_h", _l)]


_bound = None


def _lib():
    """The library, with the argument types of these entry points set once."""
    global _bound
    if _bound is None:
        lib = load_library()
        P = ctypes.POINTER
        sigs = {
            "gdr_linear_scan_fwd": [_p] * 6 + [P(gdr_scan_dims), _p],
            "gdr_linear_scan_bwd": [_p] * 8 + [P(gdr_scan_dims), _p],
            "gdr_qk_norm_rope": [_p] * 9 + [P(gdr_qk_dims), _p],
            "gdr_qk_norm_rope_bwd": [_p] * 13 + [P(gdr_qk_dims), _p, _z, _p],
            "gdr_qk_norm_rope_append": [_p] * 12 + [P(gdr_qk_dims), P(gdr_paged_cache), _p],
            "gdr_paged_decode_attn": [_p] * 7 + [P(gdr_attn_dims), P(gdr_paged_cache), _p, _z,
                                                 _p],
        }
        for name, args in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, _i
        sizes = {
            "gdr_linear_scan_checkpoints_size": [P(gdr_scan_dims)],
            "gdr_qk_norm_rope_bwd_workspace_size": [P(gdr_qk_dims)],
            "gdr_paged_decode_attn_workspace_size": [P(gdr_attn_dims), P(gdr_paged_cache)],
        }
        for name, args in sizes.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, _z
        _bound = lib
    return _bound


# A step of a decoder makes a few such calls per layer, each a few microseconds of GPU work:
# what they cost on the host counts. csrc/layers_host.cpp makes the same checks and the same
# C calls in one step for the ordinary case (torch's current stream, results of the default
# dtype or passed in); it answers None to everything else, and the code below takes over,
# with its messages. A C call that was made is not made again: its status, if it is not OK, is
# the answer. On a GB300's host a call of qk_norm_rope_append takes 13 us through the
# Python code and 2.5 us compiled, the launch included.
def _load_host(path):
    """The compiled calls, or None (with a warning) where they were not built for this torch or
    cannot be imported: every call then runs from Python."""
    if not os.path.exists(path):
        warnings.warn(f"{path} not built (chunkwise_gated_delta_gdr_gb300.build): the layers' "
                      "calls run from Python, with some 10 us more host time each")
        return None
    spec = importlib.util.spec_from_file_location("_layers_host", path)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"the layers' calls run from Python: {e}")
        return None
    return module


_host = None
if os.path.exists(LIB_PATH):
    load_library()
    _host = _load_host(host_path(torch.__version__))


# ------------------------------------------------------------------ shared checks
# One pass over a tensor's attributes; what is wrong is worked out only once something is.
F32 = torch.float32
_structs = {}


def _struct(cls, *values):
    """cls(*values), one object per set of values (sizes, strides and flags; the library
    only reads it)."""
    key = (cls, values)
    s = _structs.get(key)
    if s is None:
        if len(_structs) >= 4096:
            _structs.clear()
        s = cls(*values)
        for (name, _), v in zip(cls._fields_, values):
            if isinstance(v, int) and getattr(s, name) != v:
                raise ValueError(f"{name} = {v} is out of range")
        _structs[key] = s
    return s


def _code(name, t):
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _view(name, t, shape, device):
    """t: a CUDA tensor of this shape on `device`, its last dimension dense."""
    if t.shape == shape and t.device == device and (t.stride(-1) == 1 or shape[-1] == 1):
        return
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be dense in its last dimension")


def _dense(name, t, shape, device, dtype=F32):
    """The address of t: None, or a contiguous CUDA tensor of this shape and dtype on `device`."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _scratch(t, device):
    """Address and bytes of a caller's workspace: a contiguous CUDA tensor on `device`."""
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _stream(device, stream):
    """Raw handle of `stream` (default: torch's current stream of `device`)."""
    if device.type != "cuda" or device.index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors must be on the current CUDA device, got {device}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A result or scratch. For a stream that is not torch's current one it comes from that
    stream's pool, so that nothing queued elsewhere still uses its memory when the kernel
    writes it, and it goes back there only after the current stream's work, too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _raise(status, where):
    if status != GDR_OK:
        raise GdrError(status, where)


# ------------------------------------------------------------------ gated linear recurrence
def linear_scan_checkpoints(x, *, stream=None):
    """Buffer [B, ceil(T / 64), D] fp32 for linear_scan_fwd(checkpoints=...), which
    linear_scan_bwd reads. ``stream``: the one those calls are given."""
    B, T, D = x.shape
    return _empty((B, (T + SCAN_CHECKPOINT - 1) // SCAN_CHECKPOINT, D), torch.float32, x.device,
                  stream)


def linear_scan_fwd(x, g, initial_state=None, *, gated_input: bool = False,
                    output_final_state: bool = True, out_dtype=None, out=None, final_state=None,
                    checkpoints=None, stream=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + u_t on CUDA tensors.

    x, g [B,T,D] (bf16 or fp32 each; views allowed); u = x, or (1 - exp(g)) x with
    ``gated_input``. initial_state fp32 [B,D] or None; ``final_state`` may be the same
    buffer. ``checkpoints`` (linear_scan_checkpoints) is filled for linear_scan_bwd.
    Returns (h [B,T,D] of out_dtype, default x's; final_state fp32 [B,D] or None).
    Asynchronous on ``stream`` (default: torch's current stream).
    """
    if stream is None and out_dtype is None and _host is not None:
        r = _host.linear_scan_fwd(x, g, initial_state, gated_input, output_final_state, out,
                                  final_state, checkpoints)
        if r is not None:
            if type(r) is int:
                _raise(r, "gdr_linear_scan_fwd")
            return r
    shape, device = x.shape, x.device
    if len(shape) != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = shape
    raw = _stream(device, stream)
    xs, gs = x.stride(), g.stride()
    if xs[2] != 1 and D != 1:
        raise ValueError("x must be dense in its last dimension")
    _view("g", g, shape, device)
    if out is None:
        out = _empty(shape, out_dtype or x.dtype, device, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
    if final_state is None and output_final_state:
        final_state = _empty((B, D), torch.float32, device, stream)
    dims = _struct(gdr_scan_dims, B, T, D, _code("x", x), _code("g", g), _code("out", out),
                   bool(gated_input), xs[0], xs[1], gs[0], gs[1], 0, 0)
    state = (B, D)
    st = _lib().gdr_linear_scan_fwd(
        x.data_ptr(), g.data_ptr(), _dense("initial_state", initial_state, state, device),
        _dense("out", out, shape, device, out.dtype),
        _dense("final_state", final_state, state, device),
        _dense("checkpoints", checkpoints, (B, (T + SCAN_CHECKPOINT - 1) // SCAN_CHECKPOINT, D),
               device), dims, raw)
    _raise(st, "gdr_linear_scan_fwd")
    return out, final_state


def linear_scan_bwd(dh, x, g, checkpoints, d_final_state=None, *, gated_input: bool = False,
                    output_initial_state_grad: bool = True, dx=None, dg=None,
                    d_initial_state=None, stream=None):
    """Gradients of linear_scan_fwd: dh [B,T,D] (views allowed), x, g and gated_input as
    in the forward call, ``checkpoints`` as it filled them, d_final_state fp32 [B,D] or
    None. Returns (dx of x's dtype, dg of g's dtype, d_initial_state fp32 [B,D] or None).
    """
    if stream is None and _host is not None:
        r = _host.linear_scan_bwd(dh, x, g, checkpoints, d_final_state, gated_input,
                                  output_initial_state_grad, dx, dg, d_initial_state)
        if r is not None:
            if type(r) is int:
                _raise(r, "gdr_linear_scan_bwd")
            return r
    shape, device = x.shape, x.device
    if len(shape) != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = shape
    raw = _stream(device, stream)
    for name, t in (("x", x), ("g", g), ("dh", dh)):
        _view(name, t, shape, device)
    if checkpoints is None:
        raise ValueError("checkpoints of the forward call are needed")
    if dx is None:
        dx = _empty(shape, x.dtype, device, stream)
    if dg is None:
        dg = _empty(shape, g.dtype, device, stream)
    if d_initial_state is None and output_initial_state_grad:
        d_initial_state = _empty((B, D), torch.float32, device, stream)
    xs, gs, ds = x.stride(), g.stride(), dh.stride()
    dims = _struct(gdr_scan_dims, B, T, D, _code("x", x), _code("g", g), _code("dh", dh),
                   bool(gated_input), xs[0], xs[1], gs[0], gs[1], ds[0], ds[1])
    state = (B, D)
    st = _lib().gdr_linear_scan_bwd(
        dh.data_ptr(), x.data_ptr(), g.data_ptr(),
        _dense("checkpoints", checkpoints, (B, (T + SCAN_CHECKPOINT - 1) // SCAN_CHECKPOINT, D),
               device),
        _dense("d_final_state", d_final_state, state, device),
        _dense("dx", dx, shape, device, x.dtype), _dense("dg", dg, shape, device, g.dtype),
        _dense("d_initial_state", d_initial_state, state, device), dims, raw)
    _raise(st, "gdr_linear_scan_bwd")
    return dx, dg, d_initial_state


# ------------------------------------------------------------------ q/k norm and rotation
def _qk_dims(q, k, v, cos, sin, positions, eps, interleaved, out_code):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, T, heads, D]")
    B, T, HQ, D = q.shape
    HK = k.shape[2]
    device = q.device
    _view("q", q, (B, T, HQ, D), device)
    _view("k", k, (B, T, HK, D), device)
    if k.dtype != q.dtype:
        raise TypeError("q and k must have one dtype")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    R = rows = 0
    bits = 32
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos and sin must be [rows, R / 2]")
        rows, R = cos.shape[0], 2 * cos.shape[1]
        if positions is None:
            raise ValueError("positions are needed with cos and sin")
    if positions is not None:
        if positions.dtype == torch.int64:
            bits = 64
        elif positions.dtype != torch.int32:
            raise TypeError("positions must be int32 or int64")
        _dense("positions", positions, (B, T), device, positions.dtype)
    vs = (0, 0, 0)
    if v is not None:
        _view("v", v, (B, T, HK, D), device)
        if v.dtype != q.dtype:
            raise TypeError("q, k and v must have one dtype")
        vs = v.stride()
    qs, ks = q.stride(), k.stride()
    return _struct(gdr_qk_dims, B, T, HQ, HK, D, R, _code("q", q), out_code, bool(interleaved), bits,
                   rows, eps, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])


def _qk_shared(q_weight, k_weight, cos, sin, positions, D, device):
    half = None if cos is None else cos.shape
    return (_dense("q_weight", q_weight, (D,), device), _dense("k_weight", k_weight, (D,), device),
            _dense("cos", cos, half, device), _dense("sin", sin, half, device),
            None if positions is None else positions.data_ptr())


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, *,
                 eps: float = 1e-6, interleaved: bool = False, out_dtype=None, q_out=None,
                 k_out=None, stream=None):
    """RMS norm of every query and key head, then the position rotation, in one pass.

    q [B,T,HQ,D], k [B,T,HK,D] (bf16 or fp32, views allowed); q_weight, k_weight fp32 [D]
    or None (ones); cos, sin fp32 [rows, R/2], indexed by ``positions`` [B,T] (int32 or
    int64), turn the first R channels of each head: pairs (p, p + R/2), or (2p, 2p + 1)
    with ``interleaved``. Without cos and sin only the norm is taken. Returns
    (q_out, k_out) of out_dtype (default q's). A position outside the tables gives NaN.
    """
    if stream is None and out_dtype is None and _host is not None:
        r = _host.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved,
                               q_out, k_out)
        if r is not None:
            if type(r) is int:
                _raise(r, "gdr_qk_norm_rope")
            return r
    B, T, HQ, D = q.shape
    device, HK = q.device, k.shape[2]
    raw = _stream(device, stream)
    if q_out is None:
        q_out = _empty((B, T, HQ, D), out_dtype or q.dtype, device, stream)
    elif out_dtype is not None and q_out.dtype != out_dtype:
        raise TypeError(f"q_out must be {out_dtype}, got {q_out.dtype}")
    if k_out is None:
        k_out = _empty((B, T, HK, D), q_out.dtype, device, stream)
    dims = _qk_dims(q, k, None, cos, sin, positions, eps, interleaved, _code("q_out", q_out))
    st = _lib().gdr_qk_norm_rope(
        q.data_ptr(), k.data_ptr(),
        *_qk_shared(q_weight, k_weight, cos, sin, positions, D, device),
        _dense("q_out", q_out, (B, T, HQ, D), device, q_out.dtype),
        _dense("k_out", k_out, (B, T, HK, D), device, q_out.dtype), dims, raw)
    _raise(st, "gdr_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, cos=None, sin=None,
                     positions=None, *, eps: float = 1e-6, interleaved: bool = False, dq=None,
                     dk=None, output_weight_grads: bool = True, workspace=None, stream=None):
    """Gradients of qk_norm_rope: dq_out [B,T,HQ,D], dk_out [B,T,HK,D] (dense, one dtype),
    the rest as in the forward call. Returns (dq, dk, dq_weight, dk_weight): dense, of q's
    dtype, and fp32 [D] (None with output_weight_grads=False)."""
    if stream is None and _host is not None:
        r = _host.qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved,
                                   dq_out, dk_out, dq, dk, output_weight_grads, workspace)
        if r is not None:
            if type(r) is int:
                _raise(r, "gdr_qk_norm_rope_bwd")
            return r
    B, T, HQ, D = q.shape
    device, HK = q.device, k.shape[2]
    raw = _stream(device, stream)
    if dq is None:
        dq = _empty((B, T, HQ, D), q.dtype, device, stream)
    if dk is None:
        dk = _empty((B, T, HK, D), q.dtype, device, stream)
    dims = _qk_dims(q, k, None, cos, sin, positions, eps, interleaved, _code("dq_out", dq_out))
    dwq = dwk = ws = None
    ws_bytes = 0
    lib = _lib()
    if output_weight_grads:
        dwq = _empty((D,), torch.float32, device, stream)
        dwk = _empty((D,), torch.float32, device, stream)
        if workspace is None:
            size = lib.gdr_qk_norm_rope_bwd_workspace_size(dims)
            workspace = _empty((max(size, 256),), torch.uint8, device, stream)
        ws, ws_bytes = _scratch(workspace, device)
    st = lib.gdr_qk_norm_rope_bwd(
        _dense("dq_out", dq_out, (B, T, HQ, D), device, dq_out.dtype),
        _dense("dk_out", dk_out, (B, T, HK, D), device, dq_out.dtype), q.data_ptr(), k.data_ptr(),
        *_qk_shared(q_weight, k_weight, cos, sin, positions, D, device),
        _dense("dq", dq, (B, T, HQ, D), device, q.dtype),
        _dense("dk", dk, (B, T, HK, D), device, q.dtype),
        None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(), dims,
        ws, ws_bytes, raw)
    _raise(st, "gdr_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def _cache_dims(k_cache, v_cache, page_table, B, device):
    if k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("caches must be [pages, page_size, heads, D], page_table [B, max_pages]")
    shape, ps = k_cache.shape, k_cache.stride()
    if k_cache.device != device or (ps[3] != 1 and shape[3] != 1):
        _view("k_cache", k_cache, shape, device)
    if v_cache is not k_cache and (v_cache.shape != shape or v_cache.device != device):
        _view("v_cache", v_cache, shape, device)
    if v_cache.dtype != k_cache.dtype or v_cache.stride() != ps:
        raise ValueError("k_cache and v_cache must have one dtype and one layout")
    _dense("page_table", page_table, (B, page_table.shape[1]), device, torch.int32)
    return _struct(gdr_paged_cache, shape[0], shape[1], shape[2], shape[3],
                   _code("k_cache", k_cache), page_table.shape[1], ps[0], ps[1], ps[2])


def qk_norm_rope_append(q, k, v, q_weight, k_weight, cos, sin, positions, k_cache, v_cache,
                        page_table, *, eps: float = 1e-6, interleaved: bool = False,
                        out_dtype=None, q_out=None, stream=None):
    """qk_norm_rope for serving: the new keys (normed, rotated) and values go into their
    pages, in place; returns q_out [B,T,HQ,D].

    q, k, v [B,T,heads,D] (views allowed). k_cache, v_cache [pages, page_size, HK, D]
    (bf16 or fp32, any strides, both the same layout); token t of sequence b is stored at
    index positions[b, t] of its sequence, in page page_table[b, position // page_size]
    (int32 [B, max_pages]). A position or page out of range stores nothing and gives NaN
    in the token's q_out.
    """
    if stream is None and out_dtype is None and _host is not None:
        r = _host.qk_norm_rope_append(q, k, q_weight, k_weight, cos, sin, positions, eps,
                                      interleaved, v, k_cache, v_cache, page_table, q_out)
        if r is not None:
            if type(r) is int:
                _raise(r, "gdr_qk_norm_rope_append")
            return r
    B, T, HQ, D = q.shape
    device = q.device
    raw = _stream(device, stream)
    if q_out is None:
        q_out = _empty((B, T, HQ, D), out_dtype or q.dtype, device, stream)
    elif out_dtype is not None and q_out.dtype != out_dtype:
        raise TypeError(f"q_out must be {out_dtype}, got {q_out.dtype}")
    if positions is None or v is None:
        raise ValueError("positions and v are needed")
    dims = _qk_dims(q, k, v, cos, sin, positions, eps, interleaved, _code("q_out", q_out))
    cache = _cache_dims(k_cache, v_cache, page_table, B, device)
    st = _lib().gdr_qk_norm_rope_append(
        q.data_ptr(), k.data_ptr(), v.data_ptr(),
        *_qk_shared(q_weight, k_weight, cos, sin, positions, D, device),
        _dense("q_out", q_out, (B, T, HQ, D), device, q_out.dtype), k_cache.data_ptr(),
        v_cache.data_ptr(), page_table.data_ptr(), dims, cache, raw)
    _raise(st, "gdr_qk_norm_rope_append")
    return q_out


# ------------------------------------------------------------------ paged decode attention
def _attn_dims(q, k_cache, v_cache, page_table, scale, window, out_code):
    if q.dim() != 3:
        raise ValueError("q must be [B, HQ, D]")
    B, HQ, D = q.shape
    cache = _cache_dims(k_cache, v_cache, page_table, B, q.device)
    _view("q", q, (B, HQ, cache.D), q.device)
    qs = q.stride()
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    return _struct(gdr_attn_dims, B, HQ, _code("q", q), out_code, window, scale, qs[0],
                   qs[1]), cache


def paged_decode_attn_workspace_size(q, k_cache, page_table) -> int:
    """Bytes of scratch that paged_decode_attn needs for these sizes, at most (a window
    needs no more)."""
    dims, cache = _attn_dims(q, k_cache, k_cache, page_table, None, 0, GDR_F32)
    size = _lib().gdr_paged_decode_attn_workspace_size(dims, cache)
    if size == 0:
        raise GdrError(GDR_ERR_INVALID_ARG, "gdr_paged_decode_attn_workspace_size")
    return size


def paged_decode_attn(q, k_cache, v_cache, page_table, lens, *, scale: Optional[float] = None,
                      window: int = 0, out_dtype=None, out=None, lse=None, workspace=None,
                      stream=None):
    """Attention of one new token per sequence over its paged cache.

    q [B,HQ,D] (bf16 or fp32, a view allowed); caches and page_table as in
    qk_norm_rope_append, HQ a multiple of HK; lens int32 [B]: keys of each sequence, the
    new token's included. Only the last ``window`` keys count if it is positive. scale
    defaults to 1/sqrt(D). Returns (o [B,HQ,D] of out_dtype, default q's; lse fp32
    [B,HQ]). A sequence without keys gives zeros and -inf; a length or a page out of
    range gives NaN.
    """
    if stream is None and out_dtype is None and _host is not None:
        r = _host.paged_decode_attn(q, k_cache, v_cache, page_table, lens, scale, window, out, lse,
                                    workspace)
        if r is not None:
            if type(r) is int:
                _raise(r, "gdr_paged_decode_attn")
            return r
    shape, device = q.shape, q.device
    raw = _stream(device, stream)
    if out is None:
        out = _empty(shape, out_dtype or q.dtype, device, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
    dims, cache = _attn_dims(q, k_cache, v_cache, page_table, scale, window, _code("out", out))
    if lse is None:
        lse = _empty(shape[:2], torch.float32, device, stream)
    lib = _lib()
    if workspace is None:
        size = lib.gdr_paged_decode_attn_workspace_size(dims, cache)
        workspace = _empty((max(size, 256),), torch.uint8, device, stream)
    ws, ws_bytes = _scratch(workspace, device)
    st = lib.gdr_paged_decode_attn(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
        _dense("lens", lens, shape[:1], device, torch.int32),
        _dense("out", out, shape, device, out.dtype), _dense("lse", lse, shape[:2], device), dims,
        cache, ws, ws_bytes, raw)
    _raise(st, "gdr_paged_decode_attn")
    return out, lse
