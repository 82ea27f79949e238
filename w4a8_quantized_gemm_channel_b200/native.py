"""Thin ctypes binding over libw4a8.so (the C ABI declared in include/w4a8.h).

Argument marshalling only: torch tensors -> device pointers, strides and the
current CUDA stream. Every step of the layer runs in the library's kernels;
torch only allocates device memory. If the library is missing this module
raises at import time: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a8.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(6)

RELU = 0x01
OUT_F32, OUT_BF16, OUT_S32 = 0x00, 0x02, 0x04
STATIC_WEIGHTS = 0x08
PATH_AUTO, PATH_GENERIC, PATH_DECODE, PATH_TC = 0x00, 0x10, 0x20, 0x30
PATH_DECODE_RING, PATH_DECODE_REGS, PATH_DECODE_SPLIT = 0x40, 0x50, 0x60
PATH_TC_PAIR = 0x70
MAX_K = 2097152
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = range(5)
IO_F32, IO_BF16 = 0x000, 0x100
ACT_MAX_K = 131072

_OUT = {"f32": OUT_F32, "bf16": OUT_BF16, "s32": OUT_S32}
_OUT_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "s32": torch.int32}
_PATH = {"auto": PATH_AUTO, "generic": PATH_GENERIC, "decode": PATH_DECODE, "tc": PATH_TC,
         "ring": PATH_DECODE_RING, "regs": PATH_DECODE_REGS, "split": PATH_DECODE_SPLIT,
         "tc2": PATH_TC_PAIR}
_ACT = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}
_IO = {torch.float32: IO_F32, torch.bfloat16: IO_BF16}
PATH_NAMES = {v: k for k, v in _PATH.items()}

class Problem(ctypes.Structure):
    """struct w4a8_problem of include/w4a8.h."""
    _fields_ = [("X", ctypes.c_void_p), ("Wp", ctypes.c_void_p), ("sw", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("M", ctypes.c_int),
                ("K", ctypes.c_int), ("ldx", ctypes.c_int), ("ldp", ctypes.c_int), ("N", ctypes.c_int),
                ("ldy", ctypes.c_int)]


# Every symbol include/w4a8.h declares, with its ctypes signature.
_P, _I, _U, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
SIGNATURES = {
    "w4a8_packed_ld": (_I, [_I]),
    "w4a8_act_ld": (_I, [_I]),
    "w4a8_workspace_size": (_S, [_I, _I]),
    "w4_quantize_pack": (_I, [_P, _I, _I, _I, _P, _I, _P, _P]),
    "a8_quantize_rows": (_I, [_P, _I, _I, _I, _P, _I, _P, _P]),
    "w4a8_linear": (_I, [_P, _I, _I, _I, _P, _I, _P, _I, _P, _U, _P, _I, _P, _S, _P]),
    "w4a8_linear_q": (_I, [_P, _I, _I, _I, _P, _P, _I, _P, _I, _P, _U, _P, _I, _P]),
    "w4a8_linear_noalloc": (_I, [_P, _I, _I, _I, _P, _I, _P, _I, _P, _U, _P, _I, _P]),
    "w4a8_noalloc_scratch_bytes": (_S, []),
    "w4a8_amax_parts": (_I, [_I]),
    "w4a8_linear_chain": (_I, [_P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _U, _P, _I, _P, _P, _S, _P]),
    "w8a8_ld": (_I, [_I]),
    "w8_quantize": (_I, [_P, _I, _I, _I, _P, _I, _P, _P]),
    "w8a8_linear": (_I, [_P, _I, _I, _I, _P, _I, _P, _I, _P, _U, _P, _I, _P, _S, _P]),
    "w8a8_linear_q": (_I, [_P, _I, _I, _I, _P, _P, _I, _P, _I, _P, _U, _P, _I, _P]),
    "w4z_quantize_pack": (_I, [_P, _I, _I, _I, _P, _I, _P, _P, _P]),
    "w4z_workspace_size": (_S, [_I, _I, _I]),
    "w4z_linear": (_I, [_P, _I, _I, _I, _P, _I, _P, _P, _I, _P, _U, _P, _I, _P, _S, _P]),
    "w4z_linear_q": (_I, [_P, _I, _I, _I, _P, _P, _I, _P, _P, _I, _P, _U, _P, _I, _P, _S, _P]),
    "w4g_groups": (_I, [_I]),
    "w4g_quantize_pack": (_I, [_P, _I, _I, _I, _P, _I, _P, _P, _P]),
    "w4g_linear": (_I, [_P, _I, _I, _I, _P, _I, _P, _P, _I, _P, _U, _P, _I, _P, _S, _P]),
    "w4g_linear_q": (_I, [_P, _I, _I, _I, _P, _P, _I, _P, _P, _I, _P, _U, _P, _I, _P]),
    "w4a8_act_workspace_size": (_S, [_I, _I, _I, _I, _U]),
    "w4a8_grad_workspace_size": (_S, [_I, _I, _I, _I, _U]),
    "w4a8_linear_act": (_I, [_P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _U, _P, _I, _P, _I, _P, _S, _P]),
    "w4a8_glu": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _P, _P, _I, _U, _P, _I, _P, _P, _I, _P, _S, _P]),
    "w4a8_linear_act_grad": (_I, [_P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _I, _U, _P, _I, _P, _P, _S, _P]),
    "w4a8_glu_grad": (_I, [_P, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _U, _P, _I, _P, _P, _P, _S, _P]),
    "w4a8_last_path": (_U, []),
    "w4a8_last_launch_count": (_U, []),
    "w4a8_last_kernel": (ctypes.c_char_p, []),
    "w4a8_selftest_timeout": (_I, [ctypes.c_longlong, _P]),
    "w4a8_linear_grouped": (_I, [ctypes.POINTER(Problem), _I, _U, _P]),
    "w4a8_get_device_status": (_I, [_I, _P]),
    "w4a8_status_string": (ctypes.c_char_p, [_I]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libw4a8.so not found at {LIB_PATH}; build it with "
            "`python -m w4a8_quantized_gemm_channel_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class W4A8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.w4a8_status_string(status).decode()} (status {status})")


def _check(status: int, what: str):
    if status != OK:
        raise W4A8Error(status, what)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _under(stream, fn, args: dict):
    """fn(**args) with `stream` current, so that what it allocates belongs to
    the stream that uses it: a workspace of another stream's could be handed
    out again there while this one still reads it. What is returned is noted
    as used by the caller's stream too."""
    lead = next(iter(args.values()))
    if isinstance(lead, torch.Tensor) and lead.is_cuda and lead.device != stream.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {lead.device}")
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = fn(**dict(args, stream=None))
    if caller != stream:
        for t in out if isinstance(out, (tuple, list)) else (out,):
            if t is not None:
                t.record_stream(caller)
    return out


def _rowmajor(t: torch.Tensor, name: str):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return t.stride(0)


def packed_ld(k: int) -> int:
    return lib.w4a8_packed_ld(k)


def act_ld(k: int) -> int:
    return lib.w4a8_act_ld(k)


def workspace_size(m: int, k: int) -> int:
    return lib.w4a8_workspace_size(m, k)


def flags_for(relu: bool = False, out: str = "f32", path: str = "auto",
              static_weights: bool = False) -> int:
    return (RELU if relu else 0) | _OUT[out] | _PATH[path] | (STATIC_WEIGHTS if static_weights else 0)


def w4_quantize_pack(w: torch.Tensor, wp: torch.Tensor | None = None,
                     sw: torch.Tensor | None = None, stream=None):
    """W[K][N] float32 (CUDA) -> (Wp[N][ldp] uint8, sw[N] float32)."""
    if stream is not None:
        return _under(stream, w4_quantize_pack, locals())
    ldw = _rowmajor(w, "W")
    k, n = w.shape
    if wp is None:
        wp = torch.empty((n, packed_ld(k)), dtype=torch.uint8, device=w.device)
    if sw is None:
        sw = torch.empty(n, dtype=torch.float32, device=w.device)
    ldp = _rowmajor(wp, "Wp")
    _check(lib.w4_quantize_pack(_ptr(w), k, n, ldw, _ptr(wp), ldp, _ptr(sw), _stream()),
           "w4_quantize_pack")
    return wp, sw


def a8_quantize_rows(x: torch.Tensor, xq: torch.Tensor | None = None,
                     sx: torch.Tensor | None = None, stream=None):
    """X[M][K] float32 (CUDA) -> (Xq[M][ldq] int8, sx[M] float32)."""
    if stream is not None:
        return _under(stream, a8_quantize_rows, locals())
    ldx = _rowmajor(x, "X")
    m, k = x.shape
    if xq is None:
        xq = torch.empty((m, act_ld(k)), dtype=torch.int8, device=x.device)
    if sx is None:
        sx = torch.empty(m, dtype=torch.float32, device=x.device)
    ldq = _rowmajor(xq, "Xq")
    _check(lib.a8_quantize_rows(_ptr(x), m, k, ldx, _ptr(xq), ldq, _ptr(sx), _stream()),
           "a8_quantize_rows")
    return xq, sx


def _out_tensor(y, m, n, out, device):
    if y is None:
        y = torch.empty((m, n), dtype=_OUT_DTYPE[out], device=device)
    return y, _rowmajor(y, "Y")


def w4a8_linear(x: torch.Tensor, wp: torch.Tensor, sw: torch.Tensor,
                bias: torch.Tensor | None = None, relu: bool = False, out: str = "f32",
                path: str = "auto", y: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None,
                static_weights: bool = False) -> torch.Tensor:
    """Y[M][N] = dequant(quant8(X) @ unpack(Wp)^T) (+bias, ReLU) for X[M][K] float32.

    static_weights: promise that wp, sw and bias are final and not written by
    work still pending on the stream (W4A8_STATIC_WEIGHTS)."""
    if stream is not None:
        return _under(stream, w4a8_linear, locals())
    ldx = _rowmajor(x, "X")
    ldp = _rowmajor(wp, "Wp")
    m, k = x.shape
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, out, x.device)
    need = workspace_size(m, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib.w4a8_linear(_ptr(x), m, k, ldx, _ptr(wp), ldp, _ptr(sw), n, _ptr(bias),
                           flags_for(relu, out, path, static_weights), _ptr(y), ldy, _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream()),
           "w4a8_linear")
    return y


def w4a8_linear_q(xq: torch.Tensor, sx: torch.Tensor, k: int, wp: torch.Tensor,
                  sw: torch.Tensor, bias: torch.Tensor | None = None, relu: bool = False,
                  out: str = "f32", path: str = "auto", y: torch.Tensor | None = None,
                  stream=None, static_weights: bool = False) -> torch.Tensor:
    """Y from INT8 activations Xq[M][ldq] (first k bytes of each row) and sx[M]."""
    if stream is not None:
        return _under(stream, w4a8_linear_q, locals())
    ldq = _rowmajor(xq, "Xq")
    ldp = _rowmajor(wp, "Wp")
    m = xq.shape[0]
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, out, xq.device)
    _check(lib.w4a8_linear_q(_ptr(xq), m, k, ldq, _ptr(sx), _ptr(wp), ldp, _ptr(sw), n,
                             _ptr(bias), flags_for(relu, out, path, static_weights), _ptr(y), ldy,
                             _stream()),
           "w4a8_linear_q")
    return y


def amax_parts(n: int) -> int:
    return lib.w4a8_amax_parts(n)


def w4a8_linear_chain(x: torch.Tensor, wp: torch.Tensor, sw: torch.Tensor,
                      x_amax: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                      relu: bool = False, emit_amax: bool = True, path: str = "auto",
                      y: torch.Tensor | None = None, y_amax: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None,
                      static_weights: bool = False):
    """One chained Dense layer: Y[M][N] float32 as w4a8_linear, taking the
    input's per-row abs-max parts x_amax [M][parts] (or None) and returning
    (Y, y_amax) with y_amax [M][amax_parts(N)] (None if emit_amax is False)."""
    if stream is not None:
        return _under(stream, w4a8_linear_chain, locals())
    ldx = _rowmajor(x, "X")
    ldp = _rowmajor(wp, "Wp")
    m, k = x.shape
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, "f32", x.device)
    if emit_amax and y_amax is None:
        y_amax = torch.empty((m, amax_parts(n)), dtype=torch.float32, device=x.device)
    if not emit_amax:
        y_amax = None
    x_parts = 0
    if x_amax is not None:
        if x_amax.dim() != 2 or x_amax.shape[0] != m or not x_amax.is_contiguous():
            raise ValueError("x_amax must be a contiguous [M][parts] tensor")
        x_parts = x_amax.shape[1]
    need = workspace_size(m, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib.w4a8_linear_chain(_ptr(x), m, k, ldx, _ptr(x_amax), x_parts, _ptr(wp), ldp, _ptr(sw), n,
                                 _ptr(bias), flags_for(relu, "f32", path, static_weights), _ptr(y), ldy,
                                 _ptr(y_amax), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream()),
           "w4a8_linear_chain")
    return y, y_amax


def w4a8_linear_grouped(problems, relu: bool = False, out: str = "f32", stream=None,
                        static_weights: bool = False):
    """Many independent few-row linears in as few launches as possible.
    problems: list of (x, wp, sw, bias_or_None) with x [M][K] float32, M <= 4.
    Returns the list of outputs Y [M][N]."""
    if stream is not None:
        return _under(stream, w4a8_linear_grouped, locals())
    arr = (Problem * max(1, len(problems)))()
    ys = []
    for i, (x, wp, sw, bias) in enumerate(problems):
        ldx = _rowmajor(x, "X")
        ldp = _rowmajor(wp, "Wp")
        m, k = x.shape
        n = wp.shape[0]
        y, ldy = _out_tensor(None, m, n, out, x.device)
        ys.append(y)
        arr[i] = Problem(x.data_ptr(), wp.data_ptr(), sw.data_ptr(), None if bias is None else bias.data_ptr(),
                         y.data_ptr(), m, k, ldx, ldp, n, ldy)
    flags = (RELU if relu else 0) | _OUT[out] | (STATIC_WEIGHTS if static_weights else 0)
    _check(lib.w4a8_linear_grouped(arr, len(problems), flags, _stream()), "w4a8_linear_grouped")
    return ys


# the library's own figure, so Python and C cannot drift apart
NOALLOC_SCRATCH_BYTES = lib.w4a8_noalloc_scratch_bytes()


def w4a8_linear_noalloc(x: torch.Tensor, wp: torch.Tensor, sw: torch.Tensor,
                        bias: torch.Tensor | None = None, relu: bool = False, out: str = "f32",
                        path: str = "auto", y: torch.Tensor | None = None,
                        stream=None, static_weights: bool = False) -> torch.Tensor:
    """w4a8_linear without a caller workspace: the INT8 activations live in the
    library's fixed per-device scratch array (see include/w4a8.h)."""
    if stream is not None:
        return _under(stream, w4a8_linear_noalloc, locals())
    ldx = _rowmajor(x, "X")
    ldp = _rowmajor(wp, "Wp")
    m, k = x.shape
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, out, x.device)
    _check(lib.w4a8_linear_noalloc(_ptr(x), m, k, ldx, _ptr(wp), ldp, _ptr(sw), n, _ptr(bias),
                                   flags_for(relu, out, path, static_weights), _ptr(y), ldy,
                                   _stream()),
           "w4a8_linear_noalloc")
    return y


# ------------------------------------------------------------------ W8A8 ---
# The INT8 path the INT4 scheme extends: one INT8 weight code per byte
# (scale 127 / abs-max), the same activation step and epilogue.

def w8a8_ld(k: int) -> int:
    return lib.w8a8_ld(k)


def w8_quantize(w: torch.Tensor, wq: torch.Tensor | None = None,
                sw: torch.Tensor | None = None, stream=None):
    """W[K][N] float32 (CUDA) -> (Wq[N][ldw8] int8, sw[N] float32)."""
    if stream is not None:
        return _under(stream, w8_quantize, locals())
    ldw = _rowmajor(w, "W")
    k, n = w.shape
    if wq is None:
        wq = torch.empty((n, w8a8_ld(k)), dtype=torch.int8, device=w.device)
    if sw is None:
        sw = torch.empty(n, dtype=torch.float32, device=w.device)
    ldw8 = _rowmajor(wq, "Wq")
    _check(lib.w8_quantize(_ptr(w), k, n, ldw, _ptr(wq), ldw8, _ptr(sw), _stream()), "w8_quantize")
    return wq, sw


def w8a8_linear(x: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor,
                bias: torch.Tensor | None = None, relu: bool = False, out: str = "f32",
                path: str = "auto", y: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None,
                static_weights: bool = False) -> torch.Tensor:
    """Y[M][N] = dequant(quant8(X) @ Wq^T) (+bias, ReLU) for X[M][K] float32."""
    if stream is not None:
        return _under(stream, w8a8_linear, locals())
    ldx = _rowmajor(x, "X")
    ldw8 = _rowmajor(wq, "Wq")
    m, k = x.shape
    n = wq.shape[0]
    y, ldy = _out_tensor(y, m, n, out, x.device)
    need = workspace_size(m, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib.w8a8_linear(_ptr(x), m, k, ldx, _ptr(wq), ldw8, _ptr(sw), n, _ptr(bias),
                           flags_for(relu, out, path, static_weights), _ptr(y), ldy, _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream()),
           "w8a8_linear")
    return y


def w8a8_linear_q(xq: torch.Tensor, sx: torch.Tensor, k: int, wq: torch.Tensor,
                  sw: torch.Tensor, bias: torch.Tensor | None = None, relu: bool = False,
                  out: str = "f32", path: str = "auto", y: torch.Tensor | None = None,
                  stream=None, static_weights: bool = False) -> torch.Tensor:
    """Y from INT8 activations Xq[M][ldq] (first k bytes of each row) and sx[M]."""
    if stream is not None:
        return _under(stream, w8a8_linear_q, locals())
    ldq = _rowmajor(xq, "Xq")
    ldw8 = _rowmajor(wq, "Wq")
    m = xq.shape[0]
    n = wq.shape[0]
    y, ldy = _out_tensor(y, m, n, out, xq.device)
    _check(lib.w8a8_linear_q(_ptr(xq), m, k, ldq, _ptr(sx), _ptr(wq), ldw8, _ptr(sw), n,
                             _ptr(bias), flags_for(relu, out, path, static_weights), _ptr(y), ldy,
                             _stream()),
           "w8a8_linear_q")
    return y


# --------------------------------------------------- zero-point INT4 ---
# Asymmetric per-channel INT4 weights (scale 15 / range, integer zero point),
# stored as q - 8 nibbles in the W4A8 packed layout.

def w4z_quantize_pack(w: torch.Tensor, stream=None):
    """W[K][N] float32 (CUDA) -> (Wp[N][ldp] uint8, sa[N] float32, zp[N] int32)."""
    if stream is not None:
        return _under(stream, w4z_quantize_pack, locals())
    ldw = _rowmajor(w, "W")
    k, n = w.shape
    wp = torch.empty((n, packed_ld(k)), dtype=torch.uint8, device=w.device)
    sa = torch.empty(n, dtype=torch.float32, device=w.device)
    zp = torch.empty(n, dtype=torch.int32, device=w.device)
    _check(lib.w4z_quantize_pack(_ptr(w), k, n, ldw, _ptr(wp), wp.stride(0), _ptr(sa), _ptr(zp),
                                 _stream()), "w4z_quantize_pack")
    return wp, sa, zp


def _zworkspace(workspace, m, k, n, device):
    need = lib.w4z_workspace_size(m, k, n)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def w4z_linear(x: torch.Tensor, wp: torch.Tensor, sa: torch.Tensor, zp: torch.Tensor,
               bias: torch.Tensor | None = None, relu: bool = False, out: str = "f32",
               path: str = "auto", y: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None,
               static_weights: bool = False) -> torch.Tensor:
    """Y[M][N] of the zero-point layer for X[M][K] float32."""
    if stream is not None:
        return _under(stream, w4z_linear, locals())
    ldx = _rowmajor(x, "X")
    ldp = _rowmajor(wp, "Wp")
    m, k = x.shape
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, out, x.device)
    workspace, wsb = _zworkspace(workspace, m, k, n, x.device)
    _check(lib.w4z_linear(_ptr(x), m, k, ldx, _ptr(wp), ldp, _ptr(sa), _ptr(zp), n, _ptr(bias),
                          flags_for(relu, out, path, static_weights), _ptr(y), ldy, _ptr(workspace), wsb,
                          _stream()), "w4z_linear")
    return y


def w4z_linear_q(xq: torch.Tensor, sx: torch.Tensor, k: int, wp: torch.Tensor, sa: torch.Tensor,
                 zp: torch.Tensor, bias: torch.Tensor | None = None, relu: bool = False,
                 out: str = "f32", path: str = "auto", y: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None,
                 static_weights: bool = False) -> torch.Tensor:
    """The zero-point layer on INT8 activations Xq[M][ldq] and sx[M]."""
    if stream is not None:
        return _under(stream, w4z_linear_q, locals())
    ldq = _rowmajor(xq, "Xq")
    ldp = _rowmajor(wp, "Wp")
    m = xq.shape[0]
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, out, xq.device)
    workspace, wsb = _zworkspace(workspace, m, k, n, xq.device)
    _check(lib.w4z_linear_q(_ptr(xq), m, k, ldq, _ptr(sx), _ptr(wp), ldp, _ptr(sa), _ptr(zp), n, _ptr(bias),
                            flags_for(relu, out, path, static_weights), _ptr(y), ldy, _ptr(workspace), wsb,
                            _stream()), "w4z_linear_q")
    return y


# ---------------------------------------------------- group-wise INT4 ---
# Per (output channel, group of 128 k) scale and zero point; float32 outputs.

def w4g_quantize_pack(w: torch.Tensor, stream=None):
    """W[K][N] float32 (CUDA) -> (Wp[N][ldp] uint8, sa[N][ng] float32, zp[N][ng] int32)."""
    if stream is not None:
        return _under(stream, w4g_quantize_pack, locals())
    ldw = _rowmajor(w, "W")
    k, n = w.shape
    ng = lib.w4g_groups(k)
    wp = torch.empty((n, packed_ld(k)), dtype=torch.uint8, device=w.device)
    sa = torch.empty((n, ng), dtype=torch.float32, device=w.device)
    zp = torch.empty((n, ng), dtype=torch.int32, device=w.device)
    _check(lib.w4g_quantize_pack(_ptr(w), k, n, ldw, _ptr(wp), wp.stride(0), _ptr(sa), _ptr(zp),
                                 _stream()), "w4g_quantize_pack")
    return wp, sa, zp


def w4g_linear(x: torch.Tensor, wp: torch.Tensor, sa: torch.Tensor, zp: torch.Tensor,
               bias: torch.Tensor | None = None, relu: bool = False, out: str = "f32",
               path: str = "auto", y: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None,
               static_weights: bool = False) -> torch.Tensor:
    """Y[M][N] of the group-wise layer for X[M][K] float32."""
    if stream is not None:
        return _under(stream, w4g_linear, locals())
    ldx = _rowmajor(x, "X")
    ldp = _rowmajor(wp, "Wp")
    m, k = x.shape
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, out, x.device)
    need = workspace_size(m, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib.w4g_linear(_ptr(x), m, k, ldx, _ptr(wp), ldp, _ptr(sa), _ptr(zp), n, _ptr(bias),
                          flags_for(relu, out, path, static_weights), _ptr(y), ldy, _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _stream()), "w4g_linear")
    return y


def w4g_linear_q(xq: torch.Tensor, sx: torch.Tensor, k: int, wp: torch.Tensor, sa: torch.Tensor,
                 zp: torch.Tensor, bias: torch.Tensor | None = None, relu: bool = False,
                 out: str = "f32", path: str = "auto", y: torch.Tensor | None = None, stream=None,
                 static_weights: bool = False) -> torch.Tensor:
    """The group-wise layer on INT8 activations Xq[M][ldq] and sx[M]."""
    if stream is not None:
        return _under(stream, w4g_linear_q, locals())
    ldq = _rowmajor(xq, "Xq")
    ldp = _rowmajor(wp, "Wp")
    m = xq.shape[0]
    n = wp.shape[0]
    y, ldy = _out_tensor(y, m, n, out, xq.device)
    _check(lib.w4g_linear_q(_ptr(xq), m, k, ldq, _ptr(sx), _ptr(wp), ldp, _ptr(sa), _ptr(zp), n, _ptr(bias),
                            flags_for(relu, out, path, static_weights), _ptr(y), ldy, _stream()),
           "w4g_linear_q")
    return y


# ------------------------------------------------------- MLP operators ---
# The W4A8 product with bias, activation and residual in its epilogue, the
# gated feed-forward product, and the input gradients of both. Rows are all
# float32 or all bfloat16; act is "none", "relu", "silu", "gelu" or
# "gelu_tanh". Formulas and rules: include/w4a8.h. A call runs on `stream`, the
# current one by default; outputs and workspace that it allocates belong to that
# stream, and what it reads must be ready there. The calls take and return plain
# values: autograd does not record them, the gradient calls are made by hand.

# A call on few rows takes the GPU about as long as its marshalling takes the
# host, so this part keeps to plain integers and checks each fact once. Sizes
# are checked against _INT_MAX because ctypes cuts larger ones off silently.
_INT_MAX = 2 ** 31 - 1

def _mlp_flags(rows: torch.Tensor, act: str, path: str, static_weights: bool):
    """(flags, activation code) of a call on rows of this type."""
    try:
        return _IO[rows.dtype] | _PATH[path] | (STATIC_WEIGHTS if static_weights else 0), _ACT[act]
    except KeyError as e:
        raise ValueError(f"rows must be float32 or bfloat16, act one of {', '.join(_ACT)}, path one of "
                         f"{', '.join(_PATH)}; got {e}") from None


def _row_stride(t: torch.Tensor, name: str, rows: int, cols: int) -> int:
    """Row stride of a [rows][cols] tensor with unit column stride. torch gives
    no meaning to the stride of a single row or column."""
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1:
        return max(ld, cols) if ld <= _INT_MAX else cols
    if ld > _INT_MAX:
        raise ValueError(f"{name}'s row stride of {ld} elements does not fit an int")
    return ld


def _rows_in(t: torch.Tensor, name: str):
    """(rows, columns, row stride, device index) of a call's leading row tensor."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    m, n = t.shape
    if m > _INT_MAX or n > _INT_MAX:
        raise ValueError(f"{name} of shape {tuple(t.shape)}: sizes must fit an int")
    return m, n, _row_stride(t, name, m, n), t.get_device()


def _like(t: torch.Tensor | None, name: str, x: torch.Tensor, dev: int, m: int, n: int) -> int:
    """Row stride of an optional [m][n] tensor of x's type and device (0 for None)."""
    if t is None:
        return 0
    if t.dtype != x.dtype or t.get_device() != dev or t.shape != (m, n):
        raise ValueError(f"{name} must be a [{m}][{n}] {x.dtype} tensor on {x.device}")
    return _row_stride(t, name, m, n)


def _saved(g: torch.Tensor | None, u: torch.Tensor | None, x: torch.Tensor, dev: int, m: int, n: int) -> int:
    """Row stride of the gated form's saved pre-activations (0 for None); of
    single rows it may differ."""
    ldg, ldu = _like(g, "G", x, dev, m, n), _like(u, "U", x, dev, m, n)
    if ldg != ldu:
        if m > 1 or g is None or u is None:
            raise ValueError("G and U must both be given, with one row stride")
        return n
    return ldg


def _codes(wp: torch.Tensor, name: str, k: int, dev: int):
    """(N, row stride) of packed codes [N][>= ceil(k / 2)]."""
    if wp.dtype != torch.uint8 or wp.get_device() != dev or wp.dim() != 2 or wp.shape[1] < (k + 1) // 2:
        raise ValueError(f"{name} must be [N][>= {packed_ld(k)}] packed uint8 codes for K = {k} on device {dev}")
    n, cols = wp.shape
    if n > _INT_MAX or k > _INT_MAX:
        raise ValueError(f"{name}: N = {n}, K = {k} must fit an int")
    return n, _row_stride(wp, name, n, cols)


def _pair(wg, wu, k: int, dev: int):
    n, ldp = _codes(wg, "wg", k, dev)
    if _codes(wu, "wu", k, dev) != (n, ldp):
        raise ValueError("the two projections must have the same shape and row stride")
    return n, ldp


def _vector(t: torch.Tensor | None, name: str, n: int, dev: int) -> int | None:
    """Address of a float32 vector of n values (None for None)."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} values on device {dev}")
    return t.data_ptr()


def _at(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _mlp_call(fn, what: str, x: torch.Tensor, dev: int, size, args, workspace):
    """fn(*args, workspace, bytes, stream) on the current stream of x's device."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _mlp_call(fn, what, x, dev, size, args, workspace)
    if workspace is None:
        workspace = torch.empty(max(size(), 1), dtype=torch.uint8, device=x.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {x.device}")
    status = fn(*args, workspace.data_ptr(), workspace.nbytes, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise W4A8Error(status, what)


def act_workspace_size(m: int, k: int, n: int, projections: int = 1, dtype=torch.float32) -> int:
    return lib.w4a8_act_workspace_size(m, k, n, projections, _IO[dtype])


def grad_workspace_size(m: int, k: int, n: int, projections: int = 1, dtype=torch.float32) -> int:
    return lib.w4a8_grad_workspace_size(m, k, n, projections, _IO[dtype])


def w4a8_linear_act(x: torch.Tensor, wp: torch.Tensor, sw: torch.Tensor, bias: torch.Tensor | None = None,
                    act: str = "none", residual: torch.Tensor | None = None, save: bool = False,
                    path: str = "auto", y: torch.Tensor | None = None, z: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None, static_weights: bool = False):
    """Y[M][N] = act(dequant(quant8(X) @ unpack(Wp)^T) + bias) + residual, of
    X's dtype. With save (or z given) returns (Y, Z), Z the pre-activations
    that w4a8_linear_act_grad reads. y may be the residual itself."""
    if stream is not None:
        return _under(stream, w4a8_linear_act, locals())
    flags, code = _mlp_flags(x, act, path, static_weights)
    m, k, ldx, dev = _rows_in(x, "X")
    n, ldp = _codes(wp, "wp", k, dev)
    y, ldy = (x.new_empty((m, n)), n) if y is None else (y, _like(y, "Y", x, dev, m, n))
    z, ldz = (x.new_empty((m, n)), n) if save and z is None else (z, _like(z, "Z", x, dev, m, n))
    ldr = _like(residual, "residual", x, dev, m, n)
    _mlp_call(lib.w4a8_linear_act, "w4a8_linear_act", x, dev, lambda: act_workspace_size(m, k, n, 1, x.dtype),
              (x.data_ptr(), m, k, ldx, wp.data_ptr(), ldp, _vector(sw, "sw", n, dev), n,
               _vector(bias, "bias", n, dev), code, _at(residual), ldr, flags, y.data_ptr(), ldy, _at(z), ldz),
              workspace)
    return y if z is None else (y, z)


def w4a8_glu(x: torch.Tensor, wg: torch.Tensor, sg: torch.Tensor, wu: torch.Tensor, su: torch.Tensor,
             gate_bias: torch.Tensor | None = None, up_bias: torch.Tensor | None = None, act: str = "silu",
             save: bool = False, path: str = "auto", h: torch.Tensor | None = None,
             g: torch.Tensor | None = None, u: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None, static_weights: bool = False):
    """H[M][N] = act(G) * U of X's dtype, G and U the gate and up projections
    of X with their biases. With save (or g and u given) returns (H, G, U) for
    w4a8_glu_grad."""
    if stream is not None:
        return _under(stream, w4a8_glu, locals())
    flags, code = _mlp_flags(x, act, path, static_weights)
    m, k, ldx, dev = _rows_in(x, "X")
    n, ldp = _pair(wg, wu, k, dev)
    h, ldh = (x.new_empty((m, n)), n) if h is None else (h, _like(h, "H", x, dev, m, n))
    if save and g is None and u is None:
        g, u = x.new_empty((m, n)), x.new_empty((m, n))
    ldg = _saved(g, u, x, dev, m, n)
    _mlp_call(lib.w4a8_glu, "w4a8_glu", x, dev, lambda: act_workspace_size(m, k, n, 2, x.dtype),
              (x.data_ptr(), m, k, ldx, wg.data_ptr(), _vector(sg, "sg", n, dev), wu.data_ptr(),
               _vector(su, "su", n, dev), ldp, n, _vector(gate_bias, "gate_bias", n, dev),
               _vector(up_bias, "up_bias", n, dev), code, flags, h.data_ptr(), ldh, _at(g), _at(u), ldg),
              workspace)
    return h if g is None else (h, g, u)


def w4a8_linear_act_grad(dy: torch.Tensor, wp: torch.Tensor, sw: torch.Tensor, k: int, act: str = "none",
                         z: torch.Tensor | None = None, bias_grad: bool = False, path: str = "auto",
                         dx: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
                         static_weights: bool = False):
    """dX[M][k] (and with bias_grad dbias[N]) of w4a8_linear_act, of dY's
    dtype; z is the saved pre-activations (not needed without activation).
    The residual's gradient is dY."""
    if stream is not None:
        return _under(stream, w4a8_linear_act_grad, locals())
    flags, code = _mlp_flags(dy, act, path, static_weights)
    m, n, lddy, dev = _rows_in(dy, "dY")
    rows, ldp = _codes(wp, "wp", k, dev)
    if rows != n:
        raise ValueError(f"dY must have {rows} columns")
    if act == "none":
        z = None
    dx, lddx = (dy.new_empty((m, k)), k) if dx is None else (dx, _like(dx, "dX", dy, dev, m, k))
    ldz = _like(z, "Z", dy, dev, m, n)
    db = torch.empty(n, dtype=torch.float32, device=dy.device) if bias_grad else None
    _mlp_call(lib.w4a8_linear_act_grad, "w4a8_linear_act_grad", dy, dev,
              lambda: grad_workspace_size(m, k, n, 1, dy.dtype),
              (dy.data_ptr(), m, n, lddy, _at(z), ldz, wp.data_ptr(), ldp, _vector(sw, "sw", n, dev), k, code, flags,
               dx.data_ptr(), lddx, _at(db)), workspace)
    return (dx, db) if bias_grad else dx


def w4a8_glu_grad(dh: torch.Tensor, g: torch.Tensor, u: torch.Tensor, wg: torch.Tensor, sg: torch.Tensor,
                  wu: torch.Tensor, su: torch.Tensor, k: int, act: str = "silu", bias_grad: bool = False,
                  path: str = "auto", dx: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None, static_weights: bool = False):
    """dX[M][k] (and with bias_grad the two bias gradients [N]) of w4a8_glu,
    of dH's dtype, from the saved G and U."""
    if stream is not None:
        return _under(stream, w4a8_glu_grad, locals())
    flags, code = _mlp_flags(dh, act, path, static_weights)
    m, n, lddh, dev = _rows_in(dh, "dH")
    rows, ldp = _pair(wg, wu, k, dev)
    if rows != n:
        raise ValueError(f"dH must have {rows} columns")
    dx, lddx = (dh.new_empty((m, k)), k) if dx is None else (dx, _like(dx, "dX", dh, dev, m, k))
    if g is None:
        raise ValueError("G and U must both be given, with one row stride")
    ldg = _saved(g, u, dh, dev, m, n)
    dbg, dbu = (torch.empty(n, dtype=torch.float32, device=dh.device) if bias_grad else None for _ in range(2))
    _mlp_call(lib.w4a8_glu_grad, "w4a8_glu_grad", dh, dev, lambda: grad_workspace_size(m, k, n, 2, dh.dtype),
              (dh.data_ptr(), m, n, lddh, g.data_ptr(), u.data_ptr(), ldg, wg.data_ptr(), _vector(sg, "sg", n, dev),
               wu.data_ptr(), _vector(su, "su", n, dev), ldp, k, code, flags, dx.data_ptr(), lddx, _at(dbg),
               _at(dbu)), workspace)
    return (dx, dbg, dbu) if bias_grad else dx


def last_path() -> str:
    return PATH_NAMES.get(lib.w4a8_last_path(), "none")


def last_launch_count() -> int:
    return lib.w4a8_last_launch_count()


def last_kernel() -> str:
    """Name of the product kernel of this thread's last call ("" if none)."""
    return lib.w4a8_last_kernel().decode()


def selftest_timeout(cycles: int = 1_000_000, stream=None):
    """Enqueue the bounded-wait self-test (see include/w4a8.h)."""
    _check(lib.w4a8_selftest_timeout(cycles, _stream(stream)), "w4a8_selftest_timeout")


def get_device_status(clear: bool = False, stream=None) -> int:
    return lib.w4a8_get_device_status(int(clear), _stream(stream))
