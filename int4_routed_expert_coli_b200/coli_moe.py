"""Python binding of libcoli_moe.so (the C ABI in include/coli_moe.h).

Argument marshalling only: every function here passes device pointers,
sizes and a CUDA stream handle to the C ABI of the same name; all the work
runs in the library's kernels.  PyTorch supplies device memory and streams.

The library is loaded from this package directory; if it is missing, import
of this module raises (build it with ``python -m
int4_routed_expert_coli_b200.build``).  There is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcoli_moe.so")

# coli_status codes (include/coli_moe.h)
COLI_OK = 0
COLI_ERR_INVALID_ARG = 1
COLI_ERR_SHAPE = 2
COLI_ERR_ALIGN = 3
COLI_ERR_WORKSPACE = 4
COLI_ERR_CUDA = 5
COLI_ERR_TIMEOUT = 6
COLI_ERR_UNSUPPORTED = 7
COLI_ERR_BAD_INDEX = 8
COLI_ERR_RANGE = 9
COLI_OUT_F32 = 0
COLI_WS_LOGITS_OFFSET = 16384  # router logits left in the workspace by coli_moe_layer
COLI_WS_HEADER_BYTES = 16384
COLI_OUT_BF16 = 1
COLI_GROUP_PER_ROW = 0  # coli_moe_desc.group_size of the per-row int4 format
COLI_GATE_NONE = 0      # gate_kind of coli_moe_block_norm: no gate,
COLI_GATE_CHANNEL = 1   # one value per channel [H],
COLI_GATE_TOKEN = 2     # one value per token [T]

EXPORTS = ("coli_moe_create", "coli_moe_destroy", "coli_moe_workspace_size",
           "coli_moe_workspace_clear", "coli_moe_route", "coli_moe_union",
           "coli_moe_union_workspace_size", "coli_moe_ffn",
           "coli_moe_layer", "coli_moe_layer_noalloc", "coli_moe_combine_rows",
           "coli_moe_prefetch",
           "coli_moe_block_norm", "coli_moe_block_norm_backward",
           "coli_moe_block_norm_workspace_size",
           "coli_moe_grouped_mm", "coli_moe_grouped_mm_dx", "coli_moe_grouped_mm_dw",
           "coli_moe_grouped_workspace_size",
           "coli_moe_fp8_quantize_rows", "coli_moe_fp8_grouped_mm",
           "coli_moe_get_status",
           "coli_moe_debug_inject",
           "coli_moe_profile_enable",
           "coli_moe_profile_read", "coli_status_string")


class ColiError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class CExpert(ctypes.Structure):
    _fields_ = [("gate_q", ctypes.c_void_p), ("up_q", ctypes.c_void_p),
                ("down_q", ctypes.c_void_p), ("gate_s", ctypes.c_void_p),
                ("up_s", ctypes.c_void_p), ("down_s", ctypes.c_void_p)]


class CDesc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_routed", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("experts", ctypes.POINTER(CExpert)), ("prefill_min_tokens", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m int4_routed_expert_coli_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    L.coli_moe_create.argtypes = [ctypes.POINTER(CDesc), ctypes.POINTER(P)]
    L.coli_moe_create.restype = ctypes.c_int
    L.coli_moe_destroy.argtypes = [P]
    L.coli_moe_destroy.restype = None
    L.coli_moe_workspace_size.argtypes = [P, i32]
    L.coli_moe_workspace_size.restype = sz
    L.coli_moe_workspace_clear.argtypes = [P, sz, P]
    L.coli_moe_workspace_clear.restype = ctypes.c_int
    L.coli_moe_route.argtypes = [i32, i32, i32, P, P, P, P]
    L.coli_moe_route.restype = ctypes.c_int
    L.coli_moe_union.argtypes = [i32, i32, i32, P, P, P, P, P, P, P, sz, P]
    L.coli_moe_union.restype = ctypes.c_int
    L.coli_moe_union_workspace_size.argtypes = [i32, i32, i32]
    L.coli_moe_union_workspace_size.restype = sz
    L.coli_moe_ffn.argtypes = [P, i32, P, P, P, P, P, P, P, P, P, ctypes.c_int, P, sz, P]
    L.coli_moe_ffn.restype = ctypes.c_int
    L.coli_moe_layer.argtypes = [P, i32, P, P, P, P, P, ctypes.c_int, P, P, P, sz, P]
    L.coli_moe_layer.restype = ctypes.c_int
    L.coli_moe_layer_noalloc.argtypes = [ctypes.POINTER(CDesc), i32, P, P, P, P, ctypes.c_int, P, P]
    L.coli_moe_layer_noalloc.restype = ctypes.c_int
    L.coli_moe_combine_rows.argtypes = [i32, i32, i32, P, P, P, P, ctypes.c_int, P]
    L.coli_moe_combine_rows.restype = ctypes.c_int
    L.coli_moe_prefetch.argtypes = [P, i32, i32, P, sz, P, sz, P]
    L.coli_moe_prefetch.restype = ctypes.c_int
    f32, ci = ctypes.c_float, ctypes.c_int
    L.coli_moe_block_norm.argtypes = [i32, i32, P, ci, P, ci, P, P, i32, f32, P, f32, P, P, ci, P]
    L.coli_moe_block_norm.restype = ctypes.c_int
    L.coli_moe_block_norm_workspace_size.argtypes = [i32, i32]
    L.coli_moe_block_norm_workspace_size.restype = sz
    L.coli_moe_block_norm_backward.argtypes = [i32, i32, P, ci, P, P, ci, P, ci, P, P, i32, f32, P,
                                               f32, P, P, P, P, P, P, sz, P]
    L.coli_moe_block_norm_backward.restype = ctypes.c_int
    L.coli_moe_grouped_workspace_size.argtypes = [i32, i32]
    L.coli_moe_grouped_workspace_size.restype = sz
    L.coli_moe_grouped_mm.argtypes = [i32, i32, i32, i32, P, P, P, P, ci, P, sz, P]
    L.coli_moe_grouped_mm.restype = ctypes.c_int
    L.coli_moe_grouped_mm_dx.argtypes = [i32, i32, i32, i32, P, P, P, P, ci, P, sz, P]
    L.coli_moe_grouped_mm_dx.restype = ctypes.c_int
    L.coli_moe_grouped_mm_dw.argtypes = [i32, i32, i32, i32, P, P, P, P, ci, i32, P, sz, P]
    L.coli_moe_grouped_mm_dw.restype = ctypes.c_int
    L.coli_moe_fp8_quantize_rows.argtypes = [i32, i32, P, ci, P, P, P]
    L.coli_moe_fp8_quantize_rows.restype = ctypes.c_int
    L.coli_moe_fp8_grouped_mm.argtypes = [i32, i32, i32, i32, P, P, P, P, P, P, ci, P, sz, P]
    L.coli_moe_fp8_grouped_mm.restype = ctypes.c_int
    L.coli_moe_get_status.argtypes = [P, P]
    L.coli_moe_get_status.restype = ctypes.c_int
    L.coli_moe_debug_inject.argtypes = [i32]
    L.coli_moe_debug_inject.restype = ctypes.c_int
    L.coli_moe_profile_enable.argtypes = [i32]
    L.coli_moe_profile_enable.restype = ctypes.c_int
    L.coli_moe_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i32)]
    L.coli_moe_profile_read.restype = ctypes.c_int
    L.coli_status_string.argtypes = [ctypes.c_int]
    L.coli_status_string.restype = ctypes.c_char_p
    return L


lib = _load()


def status_string(s: int) -> str:
    return lib.coli_status_string(int(s)).decode()


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(status: int, where: str, raise_on_error: bool):
    if raise_on_error and status != COLI_OK:
        raise ColiError(status, where)
    return status


# ---- the ABI, one function each -------------------------------------------

def coli_moe_route(T, E, k, logits, topk_idx, topk_w, stream=None, raise_on_error=True):
    s = lib.coli_moe_route(T, E, k, _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _stream(stream))
    return _check(s, "coli_moe_route", raise_on_error)


def coli_moe_union(T, E, k, topk_idx, counts, offsets, pairs, active, n_active, ws=None,
                   stream=None, raise_on_error=True):
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    s = lib.coli_moe_union(T, E, k, _ptr(topk_idx), _ptr(counts), _ptr(offsets), _ptr(pairs),
                           _ptr(active), _ptr(n_active), _ptr(ws), ws_bytes, _stream(stream))
    return _check(s, "coli_moe_union", raise_on_error)


def coli_moe_union_workspace_size(T, E, k):
    return int(lib.coli_moe_union_workspace_size(T, E, k))


def coli_moe_ffn(handle, T, x, topk_w, counts, offsets, pairs, active, n_active, residual, out,
                 out_dtype, ws, stream=None, raise_on_error=True):
    s = lib.coli_moe_ffn(handle, T, _ptr(x), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                         _ptr(pairs), _ptr(active), _ptr(n_active), _ptr(residual), _ptr(out),
                         out_dtype, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    return _check(s, "coli_moe_ffn", raise_on_error)


def coli_moe_layer(handle, T, x, logits, router_w, residual, out, out_dtype, topk_idx_out, topk_w_out,
                   ws, stream=None, raise_on_error=True):
    s = lib.coli_moe_layer(handle, T, _ptr(x), _ptr(logits), _ptr(router_w), _ptr(residual),
                           _ptr(out), out_dtype, _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(ws),
                           ws.numel() * ws.element_size(), _stream(stream))
    return _check(s, "coli_moe_layer", raise_on_error)


def coli_moe_layer_noalloc(desc, T, x, logits, residual, out, out_dtype, status_out=None,
                           stream=None, raise_on_error=True):
    """Layer step without handle or workspace (see include/coli_moe.h):
    `desc` is a CDesc (e.g. MoELayer.desc), T <= 8."""
    s = lib.coli_moe_layer_noalloc(ctypes.byref(desc), T, _ptr(x), _ptr(logits), _ptr(residual),
                                   _ptr(out), out_dtype, _ptr(status_out), _stream(stream))
    return _check(s, "coli_moe_layer_noalloc", raise_on_error)


def coli_moe_combine_rows(T, k, H, rows, shared, residual, out, out_dtype, stream=None,
                          raise_on_error=True):
    s = lib.coli_moe_combine_rows(T, k, H, _ptr(rows), _ptr(shared), _ptr(residual), _ptr(out),
                                  out_dtype, _stream(stream))
    return _check(s, "coli_moe_combine_rows", raise_on_error)


def coli_moe_prefetch(handle, T, k, topk_idx, max_bytes, ws=None, stream=None,
                      raise_on_error=True):
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    s = lib.coli_moe_prefetch(handle, T, k, _ptr(topk_idx), int(max_bytes), _ptr(ws), ws_bytes,
                              _stream(stream))
    return _check(s, "coli_moe_prefetch", raise_on_error)


def coli_moe_workspace_clear(ws, stream=None, raise_on_error=True):
    s = lib.coli_moe_workspace_clear(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    return _check(s, "coli_moe_workspace_clear", raise_on_error)


def coli_moe_get_status(ws, stream=None):
    return lib.coli_moe_get_status(_ptr(ws), _stream(stream))


COLI_INJECT_WITHHOLD_STAGE = 1
COLI_INJECT_NOT_RESIDENT = 2
COLI_INJECT_WITHHOLD_GROUPED = 3
COLI_INJECT_SHORT_WAITS = 4


def coli_moe_debug_inject(what: int):
    return lib.coli_moe_debug_inject(int(what))


def coli_moe_profile_enable(enable: bool):
    return lib.coli_moe_profile_enable(1 if enable else 0)


def coli_moe_profile_read():
    """Summed milliseconds per phase [prep, gate/up, down, combine] and the
    number of recorded calls since the last read."""
    ms = (ctypes.c_double * 4)()
    n = ctypes.c_int32()
    s = lib.coli_moe_profile_read(ms, ctypes.byref(n))
    _check(s, "coli_moe_profile_read", True)
    return list(ms), int(n.value)


# ---- around the layer: norms and grouped products ---------------------------
# These functions know every argument's size, so they also check the tensors'
# types, element counts and device before any pointer is passed, and run on
# the device of their tensors (its current stream by default).

_DTYPE = {torch.float32: COLI_OUT_F32, torch.bfloat16: COLI_OUT_BF16}


def _arg(t, name, numel, dtypes, device, optional=False):
    """Address of a checked tensor argument on CUDA device `device` (None for
    an absent optional one)."""
    if t is None and optional:
        return None
    try:  # one pass over what a right argument satisfies
        if (t.get_device() == device and t.dtype in dtypes and t.numel() == numel
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if t is None:
        raise ValueError(f"{name} is missing")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the CUDA device")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, other arguments on cuda:{device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: type {t.dtype} is not one of {tuple(dtypes)}")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    raise ValueError(f"{name} has {t.numel()} elements, the call's sizes need {numel}")


_F32, _BF16, _I32 = (torch.float32,), (torch.bfloat16,), (torch.int32,)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def _int32(*sizes):
    """Sizes are passed in 32 bits: larger ones would arrive as other numbers."""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise ValueError(f"sizes {sizes} do not fit 32 bits")


def _device(*tensors):
    """Index of the CUDA device of the first tensor given."""
    for t in tensors:
        if isinstance(t, torch.Tensor):
            if not t.is_cuda:
                raise ValueError("tensor arguments must live on the CUDA device")
            return t.get_device()
    raise ValueError("no tensor argument")


def _run(fn, device, stream, *args):
    """fn(*args, stream) on `device`, by default on its current stream."""
    current = torch._C._cuda_getDevice()  # (a tensor is on a device: CUDA is set up)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    else:
        handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if device == current:
        return fn(*args, handle)
    with torch.cuda.device(device):
        return fn(*args, handle)


def _ws_arg(ws, device):
    """(pointer, bytes) of a workspace tensor of any type; (None, 0) for None."""
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws: expected a torch.Tensor")
    n = ws.numel()
    return _arg(ws, "ws", n, (ws.dtype,), device), ws.nbytes


def coli_moe_block_norm(T, H, x, y, post_w, gate, gate_kind, alpha, pre_w, eps, s_out, o,
                        stream=None, raise_on_error=True):
    """s = x + alpha * g * norm(y) post_w;  o = norm(s) pre_w (include/coli_moe.h).
    x and s_out share one type, y and o have their own (fp32 or bf16)."""
    _int32(T, H)
    dev = _device(x, s_out, o)
    n = T * H
    args = (T, H, _arg(x, "x", n, _DTYPE, dev), _DTYPE[x.dtype],
            _arg(y, "y", n, _DTYPE, dev, True), _DTYPE[y.dtype] if y is not None else 0,
            _arg(post_w, "post_w", H, _F32, dev, True),
            _arg(gate, "gate", T if gate_kind == COLI_GATE_TOKEN else H, _F32, dev, True),
            gate_kind, alpha, _arg(pre_w, "pre_w", H, _F32, dev, True), eps,
            _arg(s_out, "s_out", n, (x.dtype,), dev, True), _arg(o, "o", n, _DTYPE, dev, True),
            _DTYPE[o.dtype] if o is not None else 0)
    s = _run(lib.coli_moe_block_norm, dev, stream, *args)
    return _check(s, "coli_moe_block_norm", raise_on_error)


def coli_moe_block_norm_workspace_size(T, H):
    _int32(T, H)
    return int(lib.coli_moe_block_norm_workspace_size(T, H))


def coli_moe_block_norm_backward(T, H, d_o, d_s, s, y, post_w, gate, gate_kind, alpha, pre_w, eps,
                                 dx, dy, dpre_w, dpost_w, dgate, ws=None, stream=None,
                                 raise_on_error=True):
    """Gradients of coli_moe_block_norm from the stored s and y
    (include/coli_moe.h)."""
    _int32(T, H)
    dev = _device(d_o, d_s, s, y, dx, dy, dpre_w, dpost_w, dgate)
    n = T * H
    stream_t = next((t for t in (s, d_s, dx) if t is not None), None)
    xt = stream_t.dtype if stream_t is not None else torch.float32
    if xt not in _DTYPE:
        raise ValueError(f"type {xt} is not one of {tuple(_DTYPE)}")
    yt = y.dtype if y is not None else torch.float32
    n_gate = T if gate_kind == COLI_GATE_TOKEN else H
    ws_p, ws_n = _ws_arg(ws, dev)
    args = (T, H, _arg(d_o, "d_o", n, _DTYPE, dev, True),
            _DTYPE[d_o.dtype] if d_o is not None else 0,
            _arg(d_s, "d_s", n, (xt,), dev, True), _arg(s, "s", n, (xt,), dev, True), _DTYPE[xt],
            _arg(y, "y", n, _DTYPE, dev, True), _DTYPE[yt] if y is not None else 0,
            _arg(post_w, "post_w", H, _F32, dev, True), _arg(gate, "gate", n_gate, _F32, dev, True),
            gate_kind, alpha, _arg(pre_w, "pre_w", H, _F32, dev, True), eps,
            _arg(dx, "dx", n, (xt,), dev, True), _arg(dy, "dy", n, (yt,), dev, True),
            _arg(dpre_w, "dpre_w", H, _F32, dev, True),
            _arg(dpost_w, "dpost_w", H, _F32, dev, True),
            _arg(dgate, "dgate", n_gate, _F32, dev, True), ws_p, ws_n)
    st = _run(lib.coli_moe_block_norm_backward, dev, stream, *args)
    return _check(st, "coli_moe_block_norm_backward", raise_on_error)


def coli_moe_grouped_workspace_size(R, E):
    _int32(R, E)
    return int(lib.coli_moe_grouped_workspace_size(R, E))


def grouped_workspace(R, E, device="cuda"):
    """A cleared workspace for the grouped products of up to R rows."""
    ws = torch.empty(coli_moe_grouped_workspace_size(R, E), dtype=torch.uint8, device=device)
    with torch.cuda.device(ws.device):
        coli_moe_workspace_clear(ws)
    return ws


def coli_moe_grouped_mm(R, E, N, K, x, w, offsets, out, ws, stream=None, raise_on_error=True):
    """out[r] = w[e] x[r] for the rows of each expert (include/coli_moe.h)."""
    _int32(R, E, N, K)
    dev = _device(x, w, out)
    s = _run(lib.coli_moe_grouped_mm, dev, stream, R, E, N, K, _arg(x, "x", R * K, _BF16, dev),
             _arg(w, "w", E * N * K, _BF16, dev), _arg(offsets, "offsets", E + 1, _I32, dev),
             _arg(out, "out", R * N, _DTYPE, dev), _DTYPE[out.dtype], *_ws_arg(ws, dev))
    return _check(s, "coli_moe_grouped_mm", raise_on_error)


def coli_moe_grouped_mm_dx(R, E, N, K, dy, w, offsets, dx, ws, stream=None, raise_on_error=True):
    """dx[r] = w[e]^T dy[r] (include/coli_moe.h)."""
    _int32(R, E, N, K)
    dev = _device(dy, w, dx)
    s = _run(lib.coli_moe_grouped_mm_dx, dev, stream, R, E, N, K,
             _arg(dy, "dy", R * N, _BF16, dev), _arg(w, "w", E * N * K, _BF16, dev),
             _arg(offsets, "offsets", E + 1, _I32, dev), _arg(dx, "dx", R * K, _DTYPE, dev),
             _DTYPE[dx.dtype], *_ws_arg(ws, dev))
    return _check(s, "coli_moe_grouped_mm_dx", raise_on_error)


def coli_moe_grouped_mm_dw(R, E, N, K, dy, x, offsets, dw, accumulate, ws, stream=None,
                           raise_on_error=True):
    """dw[e] (+)= sum over the rows of e of dy[r] x[r]^T (include/coli_moe.h)."""
    _int32(R, E, N, K)
    dev = _device(dy, x, dw)
    s = _run(lib.coli_moe_grouped_mm_dw, dev, stream, R, E, N, K,
             _arg(dy, "dy", R * N, _BF16, dev), _arg(x, "x", R * K, _BF16, dev),
             _arg(offsets, "offsets", E + 1, _I32, dev), _arg(dw, "dw", E * N * K, _DTYPE, dev),
             _DTYPE[dw.dtype], 1 if accumulate else 0, *_ws_arg(ws, dev))
    return _check(s, "coli_moe_grouped_mm_dw", raise_on_error)


def coli_moe_fp8_quantize_rows(R, K, x, q, scales, stream=None, raise_on_error=True):
    """Rows to e4m3 with one fp32 scale per row and 128 values; scales is
    [ceil(K/128)][R] (include/coli_moe.h)."""
    _int32(R, K)
    dev = _device(x, q, scales)
    s = _run(lib.coli_moe_fp8_quantize_rows, dev, stream, R, K, _arg(x, "x", R * K, _DTYPE, dev),
             _DTYPE[x.dtype], _arg(q, "q", R * K, _E4M3, dev),
             _arg(scales, "scales", -(-K // 128) * R, _F32, dev))
    return _check(s, "coli_moe_fp8_quantize_rows", raise_on_error)


def coli_moe_fp8_grouped_mm(R, E, N, K, xq, x_scale, wq, w_scale, offsets, out, ws, stream=None,
                            raise_on_error=True):
    """The grouped product of e4m3 rows and weights with their block scales
    (include/coli_moe.h)."""
    _int32(R, E, N, K)
    dev = _device(xq, wq, out)
    kb = -(-K // 128)
    s = _run(lib.coli_moe_fp8_grouped_mm, dev, stream, R, E, N, K,
             _arg(xq, "xq", R * K, _E4M3, dev), _arg(x_scale, "x_scale", kb * R, _F32, dev),
             _arg(wq, "wq", E * N * K, _E4M3, dev),
             _arg(w_scale, "w_scale", E * -(-N // 128) * kb, _F32, dev),
             _arg(offsets, "offsets", E + 1, _I32, dev), _arg(out, "out", R * N, _DTYPE, dev),
             _DTYPE[out.dtype], *_ws_arg(ws, dev))
    return _check(s, "coli_moe_fp8_grouped_mm", raise_on_error)


# ---- handle ---------------------------------------------------------------

class MoELayer:
    """A coli_moe handle over an ExpertBank (device tensors; routed experts
    first, shared experts last)."""

    def __init__(self, bank, n_routed: int, top_k: int, n_shared: int = 1,
                 prefill_min_tokens: int = 0):
        """`bank.per_row` selects the per-row int4 format (group_size
        COLI_GROUP_PER_ROW) instead of gs64."""
        if bank.n != n_routed + n_shared:
            raise ValueError("bank holds a different number of experts")
        self.bank = bank
        self.H, self.I, self.E, self.k, self.n_shared = bank.hidden, bank.inter, n_routed, top_k, n_shared
        tab = (CExpert * bank.n)()
        for e in range(bank.n):
            for name in ("gate_q", "up_q", "down_q", "gate_s", "up_s", "down_s"):
                t = getattr(bank, name)[e]
                setattr(tab[e], name, t.data_ptr())
        group = COLI_GROUP_PER_ROW if getattr(bank, "per_row", False) else 64
        desc = CDesc(bank.hidden, bank.inter, n_routed, top_k, group, n_shared, tab,
                     prefill_min_tokens)
        self._table = tab
        self.desc = desc
        h = ctypes.c_void_p()
        s = lib.coli_moe_create(ctypes.byref(desc), ctypes.byref(h))
        if s != COLI_OK:
            raise ColiError(s, "coli_moe_create")
        self.handle = h

    def workspace_size(self, max_tokens: int) -> int:
        return int(lib.coli_moe_workspace_size(self.handle, max_tokens))

    def workspace(self, max_tokens: int, device=None) -> torch.Tensor:
        """A cleared workspace for calls with up to max_tokens tokens."""
        n = self.workspace_size(max_tokens)
        ws = torch.empty(n, dtype=torch.uint8, device=device or self.bank.gate_q.device)
        coli_moe_workspace_clear(ws)
        return ws

    def layer(self, x, logits=None, router_w=None, residual=None, out=None, out_dtype=COLI_OUT_F32,
              topk_idx_out=None, topk_w_out=None, ws=None, stream=None):
        T = x.shape[0]
        if out is None:
            dt = torch.float32 if out_dtype == COLI_OUT_F32 else torch.bfloat16
            out = torch.empty(T, self.H, dtype=dt, device=x.device)
        if ws is None:
            ws = self.workspace(T, x.device)
        coli_moe_layer(self.handle, T, x, logits, router_w, residual, out, out_dtype, topk_idx_out,
                       topk_w_out, ws, stream)
        return out

    def close(self):
        if getattr(self, "handle", None):
            lib.coli_moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
