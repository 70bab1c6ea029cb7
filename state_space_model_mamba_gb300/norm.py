"""Thin Python binding of the entry norm of ``libssd.so`` (``include/norm.h``):
residual addition and root-mean-square norm in one pass, with the output in
the stream's type or in e4m3 with scales, and the backward.

Argument marshalling only, as :mod:`ssd`.  ``x`` may have any number of leading
axes; its last axis is the row.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import ssd

EXPORTED = ("norm_add_rms", "norm_add_rms_fp8", "norm_backward_workspace_bytes", "norm_add_rms_backward")

_lock = threading.Lock()
_bound = None


def _lib():
    global _bound
    if _bound is not None:
        return _bound
    with _lock:
        if _bound is None:
            lib = ssd.load_library()
            vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_float
            lib.norm_add_rms.argtypes = [i32, vp, vp, vp, f32, vp, vp, i64, i64, vp]
            lib.norm_add_rms.restype = i32
            lib.norm_add_rms_fp8.argtypes = [i32, vp, vp, vp, f32, vp, vp, vp, i64, i64, i64, vp]
            lib.norm_add_rms_fp8.restype = i32
            lib.norm_backward_workspace_bytes.argtypes = [i64, i64]
            lib.norm_backward_workspace_bytes.restype = sz
            lib.norm_add_rms_backward.argtypes = [i32, vp, vp, vp, f32, vp, vp, vp, i64, i64, vp, sz, vp]
            lib.norm_add_rms_backward.restype = i32
            _bound = lib
    return _bound


# as in delta.py: addresses as plain integers, the raw stream query, messages only on failure
_BF16, _F32 = torch.bfloat16, torch.float32
_raw_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(x, weight, names, *same):
    dtype, shape, device = x.dtype, x.shape, x.device
    code = ssd.SSD_BF16 if dtype is _BF16 else ssd._dtype_code(x)
    if not shape or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor")
    D = shape[-1]
    if weight.shape != (D,) or weight.dtype is not _F32:
        raise ValueError(f"weight: expected ({D},) float32, got {tuple(weight.shape)} {weight.dtype}")
    if weight.device != device or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor on {device}")
    for i, t in enumerate(same):
        if t is not None and (t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous()):
            raise ValueError(f"{names[i]} must match x in shape, dtype and device and be contiguous")
    return code, x.numel() // max(D, 1), D, device.index


def add_rms_norm(x, weight, eps=1e-5, residual=None):
    """Returns ``(y, stream)``: stream = x + residual (x itself without a
    residual), y = stream / sqrt(mean(stream^2) + eps) * weight, both in x's type."""
    code, rows, D, index = _check(x, weight, ("residual",), residual)
    y = torch.empty_like(x)
    stream = x if residual is None else torch.empty_like(x)
    with ssd.on_device(index):
        ssd._check(_lib().norm_add_rms(code, x.data_ptr(), _ptr(residual), weight.data_ptr(), eps, y.data_ptr(),
                                       None if residual is None else _ptr(stream), rows, D, _raw_stream(index)))
    return y, stream


def add_rms_norm_fp8(x, weight, eps=1e-5, residual=None, group=0):
    """Returns ``(y8, scales, stream)``: y8 float8_e4m3fn shaped like x, scales
    fp32 [..., D / group] (group 0: one per row), y = y8 * scale."""
    code, rows, D, index = _check(x, weight, ("residual",), residual)
    y8 = torch.empty(x.shape, device=x.device, dtype=torch.float8_e4m3fn)
    scales = torch.empty(*x.shape[:-1], D // group if group else 1, device=x.device, dtype=torch.float32)
    stream = x if residual is None else torch.empty_like(x)
    with ssd.on_device(index):
        ssd._check(_lib().norm_add_rms_fp8(code, x.data_ptr(), _ptr(residual), weight.data_ptr(), eps, y8.data_ptr(),
                                           scales.data_ptr(), None if residual is None else _ptr(stream), rows, D, group,
                                           _raw_stream(index)))
    return y8, scales, stream


def add_rms_norm_backward(dy, stream, weight, eps=1e-5, d_stream=None):
    """Gradients for dy at the stored stream, with the gradient ``d_stream`` that
    reaches the stream from behind added: ``(dx, dweight)``; dx is the gradient
    of both x and residual."""
    code, rows, D, index = _check(stream, weight, ("dy", "d_stream"), dy, d_stream)
    dx = torch.empty_like(stream)
    dw = torch.empty_like(weight)
    lib = _lib()
    ws = torch.empty(lib.norm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device=stream.device)
    with ssd.on_device(index):
        ssd._check(lib.norm_add_rms_backward(code, _ptr(dy), _ptr(stream), _ptr(weight), eps, _ptr(d_stream), _ptr(dx),
                                             _ptr(dw), rows, D, _ptr(ws), ws.numel(), _raw_stream(index)))
    return dx, dw
