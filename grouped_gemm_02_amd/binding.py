"""Thin ctypes binding of libmoe.so (declared in include/moe.h).

Functions keep the C names and only marshal arguments: torch tensors become
device pointers, the current torch stream becomes the hipStream_t, and a
non-OK status becomes :class:`MoEError`. Every step of the layer runs in the
library's HIP kernels; if the library is missing this module raises, it never
falls back to another implementation.
"""
from __future__ import annotations

import array
import bisect
import ctypes
import dataclasses
import itertools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

PRECISIONS = {"bf16": 0, "fp8_block": 1, "mxfp8": 2, "fp8_bwd": 3, "fp8_fp4": 4, "fp8_block_f32": 5,
              "fp8_bwd_f32": 6}

STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_ALIGN",
    4: "MOE_ERR_PRECISION", 5: "MOE_ERR_ARCH", 6: "MOE_ERR_WORKSPACE",
    7: "MOE_ERR_LAUNCH", 8: "MOE_ERR_ROUTING", 9: "MOE_ERR_UNSUPPORTED",
}


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {moe_status_string(status)}")


MOE_FLAG_FP8_WGRAD = 1
WGRADS = {"bf16": 0, "fp8": MOE_FLAG_FP8_WGRAD}


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int64), ("k", ctypes.c_int64),
                ("precision", ctypes.c_int32), ("num_cus", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class moe_saved_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("counts", "offsets", "row_of", "src_of", "wrow", "h13", "act", "total")]


class moe_wq_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("w13", "w13_scale", "w2", "w2_scale", "w2t", "w2t_scale", "w13t", "w13t_scale", "total")]


class moe_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_double)]


MOE_DT = {"bf16": 0, "f32": 1}
# the usual quintic of the Newton-Schulz step: takes singular values in (0, 1]
# to about [0.7, 1.2] in five steps
NS_COEFFS = (3.4445, -4.7750, 2.0315)


class moe_ortho_shape(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int64), ("R", ctypes.c_int64), ("C", ctypes.c_int64),
                ("steps", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class moe_muon_params(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("mu", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("scale", ctypes.c_float), ("nesterov", ctypes.c_int32), ("reserved", ctypes.c_int32)]


MOE_SCORES = {"softmax": 0, "sigmoid": 1}
MOE_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}
MOE_STATES = {"f32": 0, "8bit": 1}
STATE_BLOCK = 128  # elements that share a scale where moments are held in 8 bits


class moe_gate_params(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("renorm", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("groups_kept", ctypes.c_int32), ("group_top", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class moe_linear_shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("act", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int64)]


class moe_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "master", "m", "v", "m_scale", "v_scale")] + \
               [("n", ctypes.c_int64), ("lr_mul", ctypes.c_float), ("decay_mul", ctypes.c_float)]


class moe_adamw_params(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state", ctypes.c_int32), ("step", ctypes.c_int64),
                ("reserved", ctypes.c_int64)]


_lib = None

_P = ctypes.c_void_p
_SIGS = {
    "moe_workspace_size": (ctypes.c_int, [ctypes.POINTER(moe_shape), ctypes.POINTER(ctypes.c_size_t),
                                          ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "moe_get_saved_layout": (ctypes.c_int, [ctypes.POINTER(moe_shape), ctypes.POINTER(moe_saved_layout)]),
    "moe_get_wq_layout": (ctypes.c_int, [ctypes.POINTER(moe_shape), ctypes.POINTER(moe_wq_layout)]),
    "moe_quantize_weights": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, _P]),
    "moe_quantize_rows": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, ctypes.c_int64, ctypes.c_int64, _P, _P,
                                         _P]),
    "moe_quantize_tokens": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, ctypes.c_int64, ctypes.c_int64, _P,
                                           _P, _P, _P, _P, _P]),
    "moe_permute_scratch_bytes": (ctypes.c_size_t, [ctypes.POINTER(moe_shape)]),
    "moe_permute": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, _P, _P, _P, _P]),
    "moe_fwd": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                               ctypes.c_size_t, _P]),
    "moe_fwd_logits": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P,
                                      _P, _P, ctypes.c_size_t, _P]),
    "moe_bwd": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                               _P, _P, ctypes.c_size_t, _P]),
    "moe_permute_noalloc": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, _P, _P, _P, _P]),
    "moe_route": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, ctypes.c_int32, _P, _P, _P]),
    "moe_route_bwd": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, _P, ctypes.c_int32, _P, _P]),
    "moe_balance_scratch_bytes": (ctypes.c_size_t, [ctypes.POINTER(moe_shape), ctypes.c_int64]),
    "moe_balance": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, ctypes.c_int64, _P, _P, _P, _P, _P, _P,
                                   _P, ctypes.c_size_t, _P]),
    "moe_balance_bwd": (ctypes.c_int, [ctypes.POINTER(moe_shape), _P, _P, _P, _P, ctypes.c_int32, _P,
                                       ctypes.c_int64, _P, _P, _P, _P, _P, _P]),
    "moe_ortho_workspace_size": (ctypes.c_int, [ctypes.POINTER(moe_ortho_shape), ctypes.POINTER(ctypes.c_size_t)]),
    "moe_orthogonalize": (ctypes.c_int, [ctypes.POINTER(moe_ortho_shape), _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_muon_step": (ctypes.c_int, [ctypes.POINTER(moe_ortho_shape), ctypes.POINTER(moe_muon_params), _P, _P, _P, _P,
                                     _P, ctypes.c_size_t, _P]),
    "moe_gate": (ctypes.c_int, [ctypes.POINTER(moe_shape), ctypes.POINTER(moe_gate_params), _P, _P, _P, _P, _P, _P]),
    "moe_gate_bwd": (ctypes.c_int, [ctypes.POINTER(moe_shape), ctypes.POINTER(moe_gate_params), _P, _P, _P,
                                    ctypes.c_int32, _P, _P]),
    "moe_linear_workspace_size": (ctypes.c_int, [ctypes.POINTER(moe_linear_shape), ctypes.POINTER(ctypes.c_size_t),
                                                 ctypes.POINTER(ctypes.c_size_t)]),
    "moe_linear": (ctypes.c_int, [ctypes.POINTER(moe_linear_shape), _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_linear_bwd": (ctypes.c_int, [ctypes.POINTER(moe_linear_shape), _P, _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "moe_adamw_step": (ctypes.c_int, [ctypes.POINTER(moe_adamw_params), ctypes.POINTER(moe_adamw_tensor),
                                      ctypes.c_int64, _P, _P, _P]),
    "moe_read_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_set_kernel_timing": (ctypes.c_int, [ctypes.c_int]),
    "moe_kernel_timing_collect": (ctypes.c_int, [ctypes.POINTER(moe_kernel_time), ctypes.c_int32,
                                                 ctypes.POINTER(ctypes.c_int32)]),
}


def lib() -> ctypes.CDLL:
    """Loads libmoe.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m grouped_gemm_02_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MoEError(status, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


MOE_ERR_SHAPE = 2


def _want(t, name: str, dtype, numel: int | None = None, optional: bool = False) -> None:
    """Checks a tensor argument before its pointer crosses the C ABI, which
    cannot see dtypes, strides or sizes: it must be a contiguous GPU tensor of
    `dtype` with at least `numel` elements. Raises MoEError(MOE_ERR_SHAPE)
    otherwise. Anything that is not a torch tensor (None, a raw address) is
    passed through for the library's own checks (NULL, alignment)."""
    if not isinstance(t, torch.Tensor):
        return
    if t.dtype != dtype:
        raise MoEError(MOE_ERR_SHAPE, f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise MoEError(MOE_ERR_SHAPE, f"{name} is not contiguous")
    if numel is not None and t.numel() < numel:
        raise MoEError(MOE_ERR_SHAPE, f"{name} holds {t.numel()} elements, needs {numel}")
    if t.device.type != "cuda":
        raise MoEError(MOE_ERR_SHAPE, f"{name} is on {t.device}, expected a GPU tensor")


def _here(stream, *wanted) -> list:
    """_want for each (tensor, name, dtype, numel), and the tensor must be on the
    current device, whose stream the call is enqueued on. Returns their
    addresses and the stream's handle."""
    dev = _current_device() if torch.cuda.is_initialized() else None  # without it there is no GPU tensor
    at = []
    for t, name, dtype, numel in wanted:
        if t is None or type(t) is int:
            at.append(t)
        elif t.get_device() == dev and t.dtype is dtype and t.numel() >= numel and t.is_contiguous():
            at.append(t.data_ptr())
        else:
            _want(t, name, dtype, numel)
            raise MoEError(MOE_ERR_SHAPE, f"{name} is on {t.device}, the current device is cuda:{dev}")
    at.append(_stream(stream) if dev is None or stream is not None else _current_handle(dev))
    return at


_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


# The handle of a device's current stream: torch's own short cut, which builds no
# Stream object, where this torch has it.
_current_handle = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda device: torch.cuda.current_stream(device).cuda_stream))


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream) -> int | None:
    if stream is None:
        if torch.cuda.is_available():
            return _current_handle(torch.cuda.current_device())
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _result(stream, sizes, dtype, device) -> torch.Tensor:
    """A result for a call on `stream`: memory of that stream, whose earlier work
    alone may still touch it, kept until what the current stream has queued by
    the time it is freed is done as well."""
    if stream is None:
        return torch.empty(*sizes, dtype=dtype, device=device)   # sizes one by one: 0.35 us less than a tuple
    device = torch.device(device)
    if device.type != "cuda":
        return torch.empty(sizes, dtype=dtype, device=device)
    here, handle = torch.cuda.current_stream(device), _stream(stream)
    if handle == here.cuda_stream:
        return torch.empty(sizes, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(sizes, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def make_shape(T, H, I, E, k, precision="bf16", num_cus=0, wgrad="bf16") -> moe_shape:
    """wgrad: "bf16" (default) or "fp8" (sets MOE_FLAG_FP8_WGRAD)."""
    p = PRECISIONS[precision] if isinstance(precision, str) else int(precision)
    f = WGRADS[wgrad] if isinstance(wgrad, str) else int(wgrad)
    return moe_shape(int(T), int(H), int(I), int(E), int(k), p, int(num_cus), f, 0)


# ------------------------------------------------------------ C entry points

def moe_status_string(status: int) -> str:
    try:
        return lib().moe_status_string(int(status)).decode()
    except RuntimeError:
        return STATUS_NAMES.get(int(status), f"status {status}")


def moe_workspace_size(shape: moe_shape):
    f, s, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_workspace_size(ctypes.byref(shape), ctypes.byref(f), ctypes.byref(s), ctypes.byref(b)),
           "moe_workspace_size")
    return f.value, s.value, b.value


def moe_get_saved_layout(shape: moe_shape) -> dict:
    out = moe_saved_layout()
    _check(lib().moe_get_saved_layout(ctypes.byref(shape), ctypes.byref(out)), "moe_get_saved_layout")
    return {n: getattr(out, n) for n, _ in moe_saved_layout._fields_}


def moe_get_wq_layout(shape: moe_shape) -> dict:
    out = moe_wq_layout()
    _check(lib().moe_get_wq_layout(ctypes.byref(shape), ctypes.byref(out)), "moe_get_wq_layout")
    return {n: getattr(out, n) for n, _ in moe_wq_layout._fields_}


def moe_quantize_weights(shape, W13, W2, wq, stream=None) -> None:
    if shape.precision != PRECISIONS["bf16"]:
        E, H, I = shape.E, shape.H, shape.I
        _want(W13, "W13", _BF16, E * 2 * I * H)
        _want(W2, "W2", _BF16, E * H * I)
        _want(wq, "wq", _U8, moe_get_wq_layout(shape)["total"])
    _check(lib().moe_quantize_weights(ctypes.byref(shape), _ptr(W13), _ptr(W2), _ptr(wq), _stream(stream)),
           "moe_quantize_weights")


def wgrad_rows_cap(shape: moe_shape) -> int:
    """K of moe_quantize_tokens' buffers: codes C*K bytes, scales C*K/32."""
    return 128 * (shape.T * shape.k // 128 + shape.E)


def moe_quantize_tokens(shape, x, ld, C, counts, offsets, src_of, codes, scales, stream=None) -> None:
    if shape.T > 0:
        K = wgrad_rows_cap(shape)
        _want(x, "in", _BF16)
        _want(counts, "counts", _I32, shape.E)
        _want(offsets, "offsets", _I32, shape.E + 1)
        _want(src_of, "src_of", _I32, shape.T * shape.k, optional=True)
        _want(codes, "codes", _U8, int(C) * K)
        _want(scales, "scales", _U8, int(C) * K // 32)
    _check(lib().moe_quantize_tokens(ctypes.byref(shape), _ptr(x), int(ld), int(C), _ptr(counts), _ptr(offsets),
                                     _ptr(src_of), _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_tokens")


def moe_quantize_rows(shape, x, rows, K, codes, scales, stream=None) -> None:
    if rows > 0:
        _want(x, "in", _BF16, int(rows) * int(K))
        _want(codes, "codes", _U8, int(rows) * int(K))
        _want(scales, "scales", _U8, int(rows) * int(K) // 32)
    _check(lib().moe_quantize_rows(ctypes.byref(shape), _ptr(x), int(rows), int(K), _ptr(codes), _ptr(scales),
                                   _stream(stream)), "moe_quantize_rows")


def moe_permute_scratch_bytes(shape: moe_shape) -> int:
    return int(lib().moe_permute_scratch_bytes(ctypes.byref(shape)))


def moe_permute(shape, topk_idx, counts, offsets, row_of, src_of, scratch, stream=None) -> None:
    Tk = shape.T * shape.k
    _want(topk_idx, "topk_idx", _I32, Tk, optional=Tk == 0)
    _want(counts, "counts", _I32, shape.E)
    _want(offsets, "offsets", _I32, shape.E + 1)
    _want(row_of, "row_of", _I32, Tk, optional=Tk == 0)
    _want(src_of, "src_of", _I32, Tk, optional=Tk == 0)
    _want(scratch, "scratch", _U8, moe_permute_scratch_bytes(shape))
    _check(lib().moe_permute(ctypes.byref(shape), _ptr(topk_idx), _ptr(counts), _ptr(offsets), _ptr(row_of),
                             _ptr(src_of), _ptr(scratch), _stream(stream)), "moe_permute")


def moe_permute_noalloc(shape, topk_idx, counts, offsets, row_of, src_of, status, stream=None) -> None:
    Tk = shape.T * shape.k
    _want(topk_idx, "topk_idx", _I32, Tk, optional=Tk == 0)
    _want(counts, "counts", _I32, shape.E)
    _want(offsets, "offsets", _I32, shape.E + 1)
    _want(row_of, "row_of", _I32, Tk, optional=Tk == 0)
    _want(src_of, "src_of", _I32, Tk, optional=Tk == 0)
    _want(status, "status", _I32, 1)
    _check(lib().moe_permute_noalloc(ctypes.byref(shape), _ptr(topk_idx), _ptr(counts), _ptr(offsets), _ptr(row_of),
                                     _ptr(src_of), _ptr(status), _stream(stream)), "moe_permute_noalloc")


def moe_fwd(shape, x, topk_idx, topk_w, W13, W2, wq, y, saved, ws, stream=None) -> None:
    T, H, I, E, k = shape.T, shape.H, shape.I, shape.E, shape.k
    f, s, _ = moe_workspace_size(shape)
    _want(x, "x", _BF16, T * H, optional=T == 0)
    _want(topk_idx, "topk_idx", _I32, T * k, optional=T == 0)
    _want(topk_w, "topk_w", _F32, T * k, optional=T == 0)
    _want(W13, "W13", _BF16, E * 2 * I * H)
    _want(W2, "W2", _BF16, E * H * I)
    _want(wq, "wq", _U8, moe_get_wq_layout(shape)["total"], optional=True)
    _want(y, "y", _BF16, T * H, optional=T == 0)
    _want(saved, "saved", _U8, s, optional=True)
    _want(ws, "ws", _U8, f)
    _check(lib().moe_fwd(ctypes.byref(shape), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(W13), _ptr(W2),
                         _ptr(wq), _ptr(y), _ptr(saved), _ptr(ws), ws.numel() * ws.element_size(),
                         _stream(stream)), "moe_fwd")


def moe_fwd_logits(shape, x, logits, renorm, topk_idx, topk_w, W13, W2, wq, y, saved, ws, stream=None) -> None:
    T, H, I, E, k = shape.T, shape.H, shape.I, shape.E, shape.k
    f, s, _ = moe_workspace_size(shape)
    _want(x, "x", _BF16, T * H, optional=T == 0)
    _want(logits, "logits", _F32, T * E, optional=T == 0)
    _want(topk_idx, "topk_idx", _I32, T * k, optional=T == 0)
    _want(topk_w, "topk_w", _F32, T * k, optional=T == 0)
    _want(W13, "W13", _BF16, E * 2 * I * H)
    _want(W2, "W2", _BF16, E * H * I)
    _want(wq, "wq", _U8, moe_get_wq_layout(shape)["total"], optional=True)
    _want(y, "y", _BF16, T * H, optional=T == 0)
    _want(saved, "saved", _U8, s, optional=True)
    _want(ws, "ws", _U8, f)
    _check(lib().moe_fwd_logits(ctypes.byref(shape), _ptr(x), _ptr(logits), int(bool(renorm)), _ptr(topk_idx),
                                _ptr(topk_w), _ptr(W13), _ptr(W2), _ptr(wq), _ptr(y), _ptr(saved), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream)), "moe_fwd_logits")


def moe_bwd(shape, dy, x, topk_idx, topk_w, W13, W2, wq, saved, dx, d_topk_w, dW13, dW2, ws,
            stream=None) -> None:
    T, H, I, E, k = shape.T, shape.H, shape.I, shape.E, shape.k
    _, s, b = moe_workspace_size(shape)
    for t, n, dt, cnt in ((dy, "dy", _BF16, T * H), (x, "x", _BF16, T * H), (topk_idx, "topk_idx", _I32, T * k),
                          (topk_w, "topk_w", _F32, T * k), (dx, "dx", _BF16, T * H),
                          (d_topk_w, "d_topk_w", _F32, T * k)):
        _want(t, n, dt, cnt, optional=T == 0)
    _want(W13, "W13", _BF16, E * 2 * I * H)
    _want(W2, "W2", _BF16, E * H * I)
    _want(wq, "wq", _U8, moe_get_wq_layout(shape)["total"], optional=True)
    _want(saved, "saved", _U8, s)
    _want(dW13, "dW13", _BF16, E * 2 * I * H)
    _want(dW2, "dW2", _BF16, E * H * I)
    _want(ws, "ws", _U8, b)
    _check(lib().moe_bwd(ctypes.byref(shape), _ptr(dy), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(W13),
                         _ptr(W2), _ptr(wq), _ptr(saved), _ptr(dx), _ptr(d_topk_w), _ptr(dW13), _ptr(dW2),
                         _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "moe_bwd")


def moe_route(shape, logits, renorm, topk_idx, topk_w, stream=None) -> None:
    if shape.T > 0:
        _want(logits, "logits", _F32, shape.T * shape.E)
        _want(topk_idx, "topk_idx", _I32, shape.T * shape.k)
        _want(topk_w, "topk_w", _F32, shape.T * shape.k)
    _check(lib().moe_route(ctypes.byref(shape), _ptr(logits), int(bool(renorm)), _ptr(topk_idx), _ptr(topk_w),
                           _stream(stream)), "moe_route")


def moe_route_bwd(shape, logits, topk_idx, topk_w, d_topk_w, renorm, d_logits, stream=None) -> None:
    if shape.T > 0:
        for t, n, dt, cnt in ((logits, "logits", _F32, shape.T * shape.E),
                              (topk_idx, "topk_idx", _I32, shape.T * shape.k),
                              (topk_w, "topk_w", _F32, shape.T * shape.k),
                              (d_topk_w, "d_topk_w", _F32, shape.T * shape.k),
                              (d_logits, "d_logits", _F32, shape.T * shape.E)):
            _want(t, n, dt, cnt)
    _check(lib().moe_route_bwd(ctypes.byref(shape), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(d_topk_w),
                               int(bool(renorm)), _ptr(d_logits), _stream(stream)), "moe_route_bwd")


def make_ortho_shape(E, R, C, steps=5, grad="bf16", coeffs=NS_COEFFS, eps=1e-7) -> moe_ortho_shape:
    """E matrices [R, C]; grad: "bf16" or "f32", the type of what is orthogonalised."""
    a, b, c = coeffs
    g = MOE_DT[grad] if isinstance(grad, str) else int(grad)
    return moe_ortho_shape(int(E), int(R), int(C), int(steps), g, float(a), float(b), float(c), float(eps),
                           0)


def moe_balance_scratch_bytes(shape: moe_shape, S: int) -> int:
    return int(lib().moe_balance_scratch_bytes(ctypes.byref(shape), int(S)))


def moe_balance(shape, logits, topk_idx, seq_offsets, S, mask, loss, counts, seq_counts, seq_probs, seq_scale, ws,
                stream=None) -> None:
    T, E, k, S = shape.T, shape.E, shape.k, int(S)
    z, idx, off, m, l, c, sc, sp, ss, w, st = _here(
        stream, (logits, "logits", _F32, T * E), (topk_idx, "topk_idx", _I32, T * k),
        (seq_offsets, "seq_offsets", _I32, S + 1), (mask, "mask", _U8, T), (loss, "loss", _F32, 2),
        (counts, "counts", _I32, E), (seq_counts, "seq_counts", _I32, S * E), (seq_probs, "seq_probs", _F32, S * E),
        (seq_scale, "seq_scale", _F32, S + 1), (ws, "ws", _U8, 0))
    _check(lib().moe_balance(ctypes.byref(shape), z, idx, off, S, m, l, c, sc, sp, ss, w, ws.numel(), st),
           "moe_balance")


def moe_balance_bwd(shape, logits, topk_idx, topk_w, d_topk_w, renorm, seq_offsets, S, mask, seq_counts, seq_scale,
                    d_loss, d_logits, stream=None) -> None:
    T, E, k, S = shape.T, shape.E, shape.k, int(S)
    z, idx, w, dw, off, m, sc, ss, dl, dz, st = _here(
        stream, (logits, "logits", _F32, T * E), (topk_idx, "topk_idx", _I32, T * k), (topk_w, "topk_w", _F32, T * k),
        (d_topk_w, "d_topk_w", _F32, T * k), (seq_offsets, "seq_offsets", _I32, S + 1), (mask, "mask", _U8, T),
        (seq_counts, "seq_counts", _I32, S * E), (seq_scale, "seq_scale", _F32, S + 1), (d_loss, "d_loss", _F32, 2),
        (d_logits, "d_logits", _F32, T * E))
    _check(lib().moe_balance_bwd(ctypes.byref(shape), z, idx, w, dw, 1 if renorm else 0, off, S, m, sc, ss, dl, dz, st),
           "moe_balance_bwd")


def moe_ortho_workspace_size(shape: moe_ortho_shape) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_ortho_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "moe_ortho_workspace_size")
    return n.value


def moe_orthogonalize(shape, G, U, ws, stream=None) -> None:
    n = shape.E * shape.R * shape.C
    g, u, w, st = _here(stream, (G, "G", _BF16 if shape.grad_dtype == 0 else _F32, n), (U, "U", _BF16, n),
                        (ws, "ws", _U8, 0))
    _check(lib().moe_orthogonalize(ctypes.byref(shape), g, u, w, ws.numel(), st), "moe_orthogonalize")


def moe_muon_step(shape, params, grad, momentum, W, master, ws, stream=None) -> None:
    n = shape.E * shape.R * shape.C
    g, m, w, ms, sp, st = _here(stream, (grad, "grad", _BF16 if shape.grad_dtype == 0 else _F32, n),
                                (momentum, "momentum", _F32, n), (W, "W", _BF16, n), (master, "master", _F32, n),
                                (ws, "ws", _U8, 0))
    _check(lib().moe_muon_step(ctypes.byref(shape), ctypes.byref(params), g, m, w, ms, sp, ws.numel(), st),
           "moe_muon_step")


def make_gate_params(score="softmax", renorm=True, groups=1, groups_kept=None, group_top=1, scale=1.0) -> moe_gate_params:
    """score: "softmax" or "sigmoid"; groups_kept defaults to all groups."""
    sc = MOE_SCORES[score] if isinstance(score, str) else int(score)
    return moe_gate_params(sc, int(bool(renorm)), int(groups), int(groups if groups_kept is None else groups_kept),
                           int(group_top), float(scale), 0)


def moe_gate(shape, params, logits, bias, mask, topk_idx, topk_w, stream=None) -> None:
    T, E, k = shape.T, shape.E, shape.k
    z, b, m, i, w, st = _here(stream, (logits, "logits", _F32, T * E), (bias, "bias", _F32, E), (mask, "mask", _U8, T),
                              (topk_idx, "topk_idx", _I32, T * k), (topk_w, "topk_w", _F32, T * k))
    _check(lib().moe_gate(ctypes.byref(shape), ctypes.byref(params), z, b, m, i, w, st), "moe_gate")


def moe_gate_bwd(shape, params, logits, topk_idx, d_topk_w, accumulate, d_logits, stream=None) -> None:
    T, E, k = shape.T, shape.E, shape.k
    z, i, w, d, st = _here(stream, (logits, "logits", _F32, T * E), (topk_idx, "topk_idx", _I32, T * k),
                           (d_topk_w, "d_topk_w", _F32, T * k), (d_logits, "d_logits", _F32, T * E))
    _check(lib().moe_gate_bwd(ctypes.byref(shape), ctypes.byref(params), z, i, w, 1 if accumulate else 0, d, st),
           "moe_gate_bwd")


def make_linear_shape(M, N, K, act="none", out="bf16") -> moe_linear_shape:
    """act: one of MOE_ACTS ("swiglu": W has 2 N rows); out: "bf16" or "f32", the type of Y, residual and dY."""
    a = MOE_ACTS[act] if isinstance(act, str) else int(act)
    o = MOE_DT[out] if isinstance(out, str) else int(out)
    return moe_linear_shape(int(M), int(N), int(K), a, o, 0)


def linear_rows(shape: moe_linear_shape) -> int:
    """N': the rows of W, the columns of P."""
    return 2 * shape.N if shape.act == MOE_ACTS["swiglu"] else shape.N


def moe_linear_workspace_size(shape: moe_linear_shape):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_linear_workspace_size(ctypes.byref(shape), ctypes.byref(f), ctypes.byref(b)),
           "moe_linear_workspace_size")
    return f.value, b.value


def moe_linear(shape, X, W, bias, residual, Y, pre, ws, stream=None) -> None:
    M, N, K, R = shape.M, shape.N, shape.K, linear_rows(shape)
    out = _BF16 if shape.out_dtype == 0 else _F32
    x, w, b, r, y, p, s, st = _here(stream, (X, "X", _BF16, M * K), (W, "W", _BF16, R * K), (bias, "bias", _F32, R),
                                    (residual, "residual", out, M * N), (Y, "Y", out, M * N), (pre, "pre", _BF16, M * R),
                                    (ws, "ws", _U8, 0))
    _check(lib().moe_linear(ctypes.byref(shape), x, w, b, r, y, p, s, 0 if ws is None else ws.numel(), st), "moe_linear")


def moe_linear_bwd(shape, dY, X, W, pre, dX, dW, dbias, ws, stream=None) -> None:
    M, N, K, R = shape.M, shape.N, shape.K, linear_rows(shape)
    out = _BF16 if shape.out_dtype == 0 else _F32
    dy, x, w, p, dx, dw, db, s, st = _here(
        stream, (dY, "dY", out, M * N), (X, "X", _BF16, M * K), (W, "W", _BF16, R * K), (pre, "pre", _BF16, M * R),
        (dX, "dX", _BF16, M * K), (dW, "dW", _BF16, R * K), (dbias, "dbias", _F32, R), (ws, "ws", _U8, 0))
    _check(lib().moe_linear_bwd(ctypes.byref(shape), dy, x, w, p, dx, dw, db, s, 0 if ws is None else ws.numel(), st),
           "moe_linear_bwd")


def moe_adamw_step(params, tensors, count, grad_scale=None, hyper=None, stream=None) -> None:
    """tensors: a ctypes array of moe_adamw_tensor (see AdamWBuffers)."""
    g, h, st = _here(stream, (grad_scale, "grad_scale", _F32, 1), (hyper, "hyper", _F32, 4))
    _check(lib().moe_adamw_step(ctypes.byref(params), tensors, int(count), g, h, st), "moe_adamw_step")


def moe_read_status(ws, stream=None) -> int:
    out = ctypes.c_int32()
    _check(lib().moe_read_status(_ptr(ws), ctypes.byref(out), _stream(stream)), "moe_read_status")
    return out.value


def moe_set_kernel_timing(enable: bool) -> None:
    _check(lib().moe_set_kernel_timing(1 if enable else 0), "moe_set_kernel_timing")


def moe_kernel_timing_collect(max_entries: int = 64) -> dict:
    arr = (moe_kernel_time * max_entries)()
    n = ctypes.c_int32()
    _check(lib().moe_kernel_timing_collect(arr, max_entries, ctypes.byref(n)), "moe_kernel_timing_collect")
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n.value)}


# ------------------------------------------------------------ buffer plumbing

@dataclasses.dataclass
class LayerBuffers:
    """Device buffers of one layer shape (allocated once with torch). `wq`
    holds the quantized weights of the FP8 precisions (None for bf16)."""
    shape: moe_shape
    fwd_ws: torch.Tensor
    saved: torch.Tensor
    bwd_ws: torch.Tensor
    layout: dict
    wq: torch.Tensor | None = None
    wq_layout: dict | None = None

    @classmethod
    def allocate(cls, shape: moe_shape, device="cuda") -> "LayerBuffers":
        f, s, b = moe_workspace_size(shape)
        mk = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device=device)  # noqa: E731
        wl = moe_get_wq_layout(shape)
        wq = mk(wl["total"]) if wl["total"] > 0 else None
        return cls(shape, mk(f), mk(s), mk(b), moe_get_saved_layout(shape), wq, wl)

    def saved_view(self, name: str, dtype, count: int) -> torch.Tensor:
        off = self.layout[name]
        esz = torch.empty((), dtype=dtype).element_size()
        return self.saved[off:off + count * esz].view(dtype)


def quantize_weights(buf: LayerBuffers, W13, W2, stream=None) -> None:
    """Refreshes buf.wq from the bf16 weights (no-op for bf16)."""
    if buf.wq is not None:
        moe_quantize_weights(buf.shape, W13, W2, buf.wq, stream)


def forward(buf: LayerBuffers, x, topk_idx, topk_w, W13, W2, y=None, training=True, stream=None):
    """Forward; for FP8 precisions buf.wq must hold quantize_weights of W13, W2."""
    s = buf.shape
    if y is None:
        y = _result(stream, (s.T, s.H), _BF16, x.device)
    moe_fwd(s, x, topk_idx, topk_w, W13, W2, buf.wq, y, buf.saved if training else None, buf.fwd_ws, stream)
    return y


def forward_logits(buf: LayerBuffers, x, logits, renorm, topk_idx, topk_w, W13, W2, y=None, training=True,
                   stream=None):
    """Forward with the router fused in: writes topk_idx and topk_w."""
    s = buf.shape
    if y is None:
        y = _result(stream, (s.T, s.H), _BF16, x.device)
    moe_fwd_logits(s, x, logits, renorm, topk_idx, topk_w, W13, W2, buf.wq, y, buf.saved if training else None,
                   buf.fwd_ws, stream)
    return y


def backward(buf: LayerBuffers, dy, x, topk_idx, topk_w, W13, W2, grads=None, stream=None):
    s = buf.shape
    if grads is None:
        dev = dy.device
        grads = (_result(stream, (s.T, s.H), _BF16, dev), _result(stream, (s.T, s.k), _F32, dev),
                 _result(stream, (s.E, 2 * s.I, s.H), _BF16, dev), _result(stream, (s.E, s.H, s.I), _BF16, dev))
    dx, dw, dW13, dW2 = grads
    moe_bwd(s, dy, x, topk_idx, topk_w, W13, W2, buf.wq, buf.saved, dx, dw, dW13, dW2, buf.bwd_ws, stream)
    return grads


@dataclasses.dataclass
class BalanceBuffers:
    """Outputs and scratch of the routing balance of one batch shape with S
    sequences (allocated once with torch; see moe_balance for their meaning)."""
    shape: moe_shape
    S: int
    loss: torch.Tensor
    counts: torch.Tensor
    seq_counts: torch.Tensor
    seq_probs: torch.Tensor
    seq_scale: torch.Tensor
    ws: torch.Tensor

    @classmethod
    def allocate(cls, shape: moe_shape, S: int = 1, device="cuda") -> "BalanceBuffers":
        E, S = shape.E, int(S)
        mk = lambda n, dt: torch.empty(n, dtype=dt, device=device)  # noqa: E731
        return cls(shape, S, mk((2,), _F32), mk((E,), _I32), mk((S, E), _I32), mk((S, E), _F32), mk((S + 1,), _F32),
                   mk((max(moe_balance_scratch_bytes(shape, S), 256),), _U8))


def balance(buf: BalanceBuffers, logits, topk_idx, seq_offsets=None, mask=None, stream=None) -> BalanceBuffers:
    """Balance loss, z-loss and counts of a routed batch, into (and as) `buf`."""
    moe_balance(buf.shape, logits, topk_idx, seq_offsets, buf.S, mask, buf.loss, buf.counts, buf.seq_counts,
                buf.seq_probs, buf.seq_scale, buf.ws, stream)
    return buf


def balance_bwd(buf: BalanceBuffers, logits, topk_idx, topk_w, d_topk_w, renorm, d_loss, seq_offsets=None, mask=None,
                seq_counts=None, seq_scale=None, d_logits=None, stream=None):
    """d_logits of the balance losses and, with d_topk_w, of the routing
    weights; seq_counts and seq_scale default to what balance left in `buf`."""
    if d_logits is None:
        d_logits = _result(stream, (buf.shape.T, buf.shape.E), _F32, buf.loss.device)
    moe_balance_bwd(buf.shape, logits, topk_idx, topk_w, d_topk_w, renorm, seq_offsets, buf.S, mask,
                    buf.seq_counts if seq_counts is None else seq_counts,
                    buf.seq_scale if seq_scale is None else seq_scale, d_loss, d_logits, stream)
    return d_logits


@dataclasses.dataclass
class OrthoBuffers:
    """Scratch of orthogonalize and muon_step for one stack of matrices."""
    shape: moe_ortho_shape
    ws: torch.Tensor

    @classmethod
    def allocate(cls, shape: moe_ortho_shape, device="cuda") -> "OrthoBuffers":
        return cls(shape, torch.empty(max(moe_ortho_workspace_size(shape), 256), dtype=_U8, device=device))


def orthogonalize(buf: OrthoBuffers, G, U=None, stream=None):
    """The orthogonalised G (bf16); U may be a bf16 G itself."""
    s = buf.shape
    if U is None:
        U = _result(stream, (s.E, s.R, s.C), _BF16, G.device)
    moe_orthogonalize(s, G, U, buf.ws, stream)
    return U


def muon_step(buf: OrthoBuffers, grad, momentum, W, *, lr, momentum_coef=0.95, weight_decay=0.0, scale=1.0,
              nesterov=True, master=None, stream=None) -> None:
    """One optimizer step on the weights W in place (see moe_muon_step)."""
    p = moe_muon_params(float(lr), float(momentum_coef), float(weight_decay), float(scale), int(bool(nesterov)), 0)
    moe_muon_step(buf.shape, p, grad, momentum, W, master, buf.ws, stream)


def gate(shape: moe_shape, params: moe_gate_params, logits, bias=None, mask=None, topk_idx=None, topk_w=None,
         stream=None):
    """(topk_idx, topk_w) of the experts chosen for each token (see moe_gate)."""
    i, w = topk_idx, topk_w
    # (addresses of results made here need no checks)
    if i is None:
        topk_idx = _result(stream, (shape.T, shape.k), _I32, logits.device)
        i = topk_idx.data_ptr()
    if w is None:
        topk_w = _result(stream, (shape.T, shape.k), _F32, logits.device)
        w = topk_w.data_ptr()
    moe_gate(shape, params, logits, bias, mask, i, w, stream)
    return topk_idx, topk_w


def gate_bwd(shape: moe_shape, params: moe_gate_params, logits, topk_idx, d_topk_w, d_logits=None, accumulate=False,
             stream=None):
    """d_logits of the chosen weights' gradient; accumulate adds to the d_logits given."""
    d = d_logits
    if d is None:
        if accumulate:
            raise MoEError(MOE_ERR_SHAPE, "accumulate needs a d_logits to add to")
        d_logits = _result(stream, (shape.T, shape.E), _F32, logits.device)
        d = d_logits.data_ptr()
    moe_gate_bwd(shape, params, logits, topk_idx, d_topk_w, accumulate, d, stream)
    return d_logits


@dataclasses.dataclass
class LinearBuffers:
    """Scratch of linear and linear_bwd for one shape; serves fewer rows too."""
    shape: moe_linear_shape
    fwd_ws: torch.Tensor
    bwd_ws: torch.Tensor | None

    @classmethod
    def allocate(cls, shape: moe_linear_shape, device="cuda", training=True) -> "LinearBuffers":
        f, b = moe_linear_workspace_size(shape)
        mk = lambda n: torch.empty(max(n, 256), dtype=_U8, device=device)  # noqa: E731
        return cls(shape, mk(f), mk(b) if training else None)

    def _of(self, X, cols: int) -> moe_linear_shape:
        s, size = self.shape, tuple(X.shape)
        if size == (s.M, cols):
            return s
        if len(size) != 2 or size[1] != cols or size[0] > s.M:
            raise MoEError(MOE_ERR_SHAPE, f"rows are {list(size)}, the buffers are for up to {s.M} of {cols}")
        return moe_linear_shape(size[0], s.N, s.K, s.act, s.out_dtype, 0)


def linear(buf: LinearBuffers, X, W, bias=None, residual=None, Y=None, pre=None, stream=None):
    """act(X W^T + bias) + residual for the rows X has (see moe_linear)."""
    s = buf._of(X, buf.shape.K)
    y = Y
    if y is None:
        Y = _result(stream, (s.M, s.N), _BF16 if s.out_dtype == 0 else _F32, X.device)
        y = Y.data_ptr()
    moe_linear(s, X, W, bias, residual, y, pre, buf.fwd_ws, stream)
    return Y


def linear_bwd(buf: LinearBuffers, dY, X, W, pre=None, bias=False, dX=None, dW=None, dbias=None, need_dX=True,
               need_dW=True, stream=None):
    """(dX, dW, dbias) of linear; dbias is None unless `bias` (or a dbias) is
    given, dX and dW are None where they are not needed."""
    s, dev = buf._of(dY, buf.shape.N), dY.device
    R = linear_rows(s)
    if dX is None and need_dX:
        dX = _result(stream, (s.M, s.K), _BF16, dev)
    if dW is None and need_dW:
        dW = _result(stream, (R, s.K), _BF16, dev)
    if dbias is None and bias:
        dbias = _result(stream, (R,), _F32, dev)
    moe_linear_bwd(s, dY, X, W, pre, dX, dW, dbias, buf.bwd_ws, stream)
    return dX, dW, dbias


_addresses = torch.Tensor.data_ptr  # with map: a fifth less than in a comprehension

# Are tensors (a list) at these addresses? Torch's own loop, where this torch has it.
_are_at = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal", None) or (
    lambda tensors, at, _: list(map(_addresses, tensors)) == at)


class _Like:
    """Do tensors have the types, devices, sizes and strides that these have? Torch's own
    comparison, one call for all of them (0.09 us a tensor; asking each for its size, type, device and
    density in Python takes 0.35). False where this torch has none, or is in another mode: then
    they are looked at one by one."""

    def __init__(self, tensors):
        try:
            from torch._C._dynamo.guards import TensorGuards
            self._guards = TensorGuards(*tensors, dynamic_dims_sizes=None, dynamic_dims_strides=None)
        except Exception:
            self._guards = None

    def __call__(self, tensors) -> bool:
        return self._guards is not None and self._guards.check(*tensors)


class AdamWBuffers:
    """The tensors of an AdamW step with their moments: lists of the parameters
    (bf16 or fp32, one type for all), m and v (fp32 of the parameter's size, or
    uint8 codes with a scale byte per 128 elements), optionally fp32 masters of bf16
    parameters (an entry may be None) and multipliers of the learning rate and the
    weight decay per tensor. It holds the tensors and looks up at every step where they
    are: one whose storage was exchanged (`t.data = loaded`) is checked anew and taken
    where it is now."""

    def __init__(self, params, m, v, m_scale=None, v_scale=None, master=None, lr_mul=None, decay_mul=None):
        n = len(params)
        none = [None] * n
        self.params, self.m, self.v = tuple(params), tuple(m), tuple(v)
        self.m_scale, self.v_scale = tuple(m_scale or none), tuple(v_scale or none)
        self.master = tuple(master or none)
        self.state = "f32" if m_scale is None else "8bit"
        self.lr_mul, self.decay_mul = tuple(lr_mul or [1.0] * n), tuple(decay_mul or [1.0] * n)
        for name in ("m", "v", "m_scale", "v_scale", "master", "lr_mul", "decay_mul"):
            if len(getattr(self, name)) != n:
                raise MoEError(MOE_ERR_SHAPE, f"{n} parameters and {len(getattr(self, name))} of {name}")
        if (m_scale is None) != (v_scale is None):
            raise MoEError(MOE_ERR_SHAPE, "m_scale and v_scale go together")
        self.dtype = self.params[0].dtype if n else _F32
        if self.dtype not in (_BF16, _F32):
            raise MoEError(MOE_ERR_SHAPE, f"parameters are {self.dtype}, expected bf16 or fp32")
        self.device = self.params[0].device if n else None
        self._sizes = [p.numel() for p in self.params]
        self._table = (moe_adamw_tensor * max(n, 1))()
        for e, k, lr, decay in zip(self._table, self._sizes, self.lr_mul, self.decay_mul):
            e.n, e.lr_mul, e.decay_mul = k, float(lr), float(decay)
        # the table's words of 8 bytes, and its columns of gradients and sizes
        words = memoryview(self._table).cast("B").cast("q")
        width = ctypes.sizeof(moe_adamw_tensor) // 8
        self._grad_words, self._size_words = (words[getattr(moe_adamw_tensor, name).offset // 8::width][:n]
                                              for name in ("grad", "n"))
        # what the step reads and writes beside parameters and gradients
        self._state = [t for ts in (self.m, self.v, self.m_scale, self.v_scale, self.master) for t in ts if t is not None]
        self._look()

    def _look(self) -> None:
        """Checks all tensors and takes their addresses."""
        mt = _F32 if self.state == "f32" else _U8
        for i, (p, k) in enumerate(zip(self.params, self._sizes)):
            b = -(-k // STATE_BLOCK)
            if p.numel() != k:
                raise MoEError(MOE_ERR_SHAPE, f"param[{i}] holds {p.numel()} elements, had {k}")
            for t, name, dt, size in ((p, "param", self.dtype, k), (self.m[i], "m", mt, k), (self.v[i], "v", mt, k),
                                      (self.m_scale[i], "m_scale", _U8, b), (self.v_scale[i], "v_scale", _U8, b),
                                      (self.master[i], "master", _F32, k)):
                if t is None and name in ("master", "m_scale", "v_scale"):
                    continue
                _want(t, f"{name}[{i}]", dt, size)
                if t.device != self.device:
                    raise MoEError(MOE_ERR_SHAPE, f"{name}[{i}] is on {t.device}, param[0] was on {self.device}")
        self._grads_at = None
        self._refuse_overlap()
        for i, e in enumerate(self._table[:len(self.params)]):
            e.param, e.m, e.v, e.master = (_ptr(t[i]) for t in (self.params, self.m, self.v, self.master))
            e.m_scale, e.v_scale = _ptr(self.m_scale[i]), _ptr(self.v_scale[i])
        self._all = [*self.params, *self._state]
        self._all_at, self._order = list(map(_addresses, self._all)), list(range(len(self._all)))
        self._params_like, self._grads_like = _Like(self.params), None
        # Other names of the moments' memory: while they live no other tensor's can be at these
        # addresses, so a moment at its address has that memory.
        self._held = [t.detach() for t in self._state]

    def _moved(self) -> bool:
        """Is a tensor no longer what was looked at?"""
        return not (_are_at(self._all, self._all_at, self._order) and self._params_like(self.params))

    def _refuse_overlap(self) -> None:
        """No buffer that a step writes may share memory with another of its buffers."""
        spans = []
        for name in ("params", "m", "v", "m_scale", "v_scale", "master"):
            spans += [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name)
                      for t in getattr(self, name) if t is not None and t.numel()]
        spans.sort()
        for a, b in zip(spans, spans[1:]):
            if b[0] < a[1]:
                raise MoEError(MOE_ERR_SHAPE, f"buffers of {a[2]} and {b[2]} overlap")
        # where they end and begin, in order, with room before the first and behind the last
        self._ends, self._starts = [0] + [s[1] for s in spans], [s[0] for s in spans] + [1 << 64]

    def _refuse_grads(self, at, sizes, dtype) -> None:
        """Nor may a gradient lie where the step writes."""
        width = dtype.itemsize
        below = map(bisect.bisect_right, itertools.repeat(self._starts), at)   # how many begin no later
        for i, (a, k, j) in enumerate(zip(at, sizes, below)):
            if k and (self._ends[j] > a or self._starts[j] < a + k * width):
                raise MoEError(MOE_ERR_SHAPE, f"grads[{i}] overlaps a buffer that the step writes")
        self._grads_at = (at, dtype)

    @classmethod
    def allocate(cls, params, state="f32", master=False, lr_mul=None, decay_mul=None) -> "AdamWBuffers":
        """Moments of zero (and fp32 copies of bf16 parameters as masters) beside the parameters."""
        params = list(params)
        if state not in MOE_STATES:
            raise MoEError(MOE_ERR_SHAPE, f"state is {state!r}, expected one of {sorted(MOE_STATES)}")
        mk = lambda p, n, dt: torch.zeros(n, dtype=dt, device=p.device)  # noqa: E731
        dt = _F32 if state == "f32" else _U8
        m, v = ([mk(p, p.numel(), dt) for p in params] for _ in range(2))
        sc = [None, None]
        if state == "8bit":
            sc = [[mk(p, -(-p.numel() // STATE_BLOCK), _U8) for p in params] for _ in range(2)]
        ms = [p.detach().float().clone().view(-1) for p in params] if master else None
        return cls(params, m, v, sc[0], sc[1], ms, lr_mul, decay_mul)


def adamw_step(buf: AdamWBuffers, grads, *, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1,
               grad_scale=None, hyper=None, stream=None) -> None:
    """One AdamW step on the parameters in place (see moe_adamw_step). grads: one tensor
    per parameter, bf16 or fp32, one type for all; None passes a parameter over."""
    n, grads = len(buf.params), list(grads)
    if len(grads) != n:
        raise MoEError(MOE_ERR_SHAPE, f"{n} parameters and {len(grads)} gradients")
    dev = _current_device() if torch.cuda.is_initialized() else None
    if n and buf.device.type == "cuda" and buf.device.index != dev:
        raise MoEError(MOE_ERR_SHAPE, f"the parameters are on {buf.device}, the current device is cuda:{dev}")
    gt = next((g.dtype for g in grads if g is not None), _F32)
    if gt not in (_BF16, _F32):
        raise MoEError(MOE_ERR_SHAPE, f"gradients are {gt}, expected bf16 or fp32")
    # all at once: a call for many small tensors is bound by these lines
    sizes, there = buf._sizes, grads
    try:
        at = list(map(_addresses, grads))
    except TypeError:   # None among them
        at = [0 if g is None else g.data_ptr() for g in grads]
        sizes = [0 if g is None else k for g, k in zip(grads, sizes)]
        there = [g for g in grads if g is not None]
    if buf._moved():
        buf._look()
    if there is not grads or buf._grads_like is None or not buf._grads_like(grads):
        want = [k for g, k in zip(grads, buf._sizes) if g is not None]
        if (list(map(torch.Tensor.numel, there)) != want or not all([t.dtype is gt for t in there])
                or not all(map(torch.Tensor.is_contiguous, there)) or any([t.get_device() != dev for t in there])):
            for i, (t, k) in enumerate(zip(there, want)):
                _want(t, f"grads[{i}]", gt, k)
                if t.numel() != k or t.get_device() != dev:
                    raise MoEError(MOE_ERR_SHAPE, f"grads[{i}] holds {t.numel()} elements on {t.device}, needs "
                                   f"{k} on cuda:{dev}")
        if there is grads:
            buf._grads_like = _Like(grads)
    if n:
        # (gradients of these addresses, sizes and type were looked over)
        if (at, gt) != buf._grads_at:
            buf._refuse_grads(at, sizes, gt)
        buf._grad_words[:], buf._size_words[:] = array.array("q", at), array.array("q", sizes)
    p = moe_adamw_params(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                         MOE_DT["bf16"] if buf.dtype is _BF16 else MOE_DT["f32"],
                         MOE_DT["bf16"] if gt is _BF16 else MOE_DT["f32"], MOE_STATES[buf.state], int(step), 0)
    moe_adamw_step(p, buf._table, n, grad_scale, hyper, stream)
