"""Thin Python binding of window attention's entry points of ``libssd.so``
(``include/window.h``): forward and backward over sequences, and for decoding the ring
of each request, filled from a prompt and stepped token by token.

Argument marshalling only, as :mod:`ssd`: torch CUDA tensors supply memory and
streams, every step runs in the library's kernels, and a missing library or a
failed call raises.  Tensors are used on the current stream of their device.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import ssd

EXPORTED = ("window_supported", "window_workspace_bytes", "window_forward", "window_backward", "window_fill", "window_step")
WINDOW_FLAG_SIMT = 1

_lock = threading.Lock()
_bound = None


class WindowDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("window", ctypes.c_int64),
                ("sinks", ctypes.c_int64), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


def _lib():
    global _bound
    if _bound is not None:
        return _bound
    with _lock:
        if _bound is None:
            lib = ssd.load_library()
            vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_float
            dims_p = ctypes.POINTER(WindowDims)
            lib.window_supported.argtypes = [dims_p, i32]
            lib.window_supported.restype = i32
            lib.window_workspace_bytes.argtypes = [dims_p, i32, i32]
            lib.window_workspace_bytes.restype = sz
            lib.window_forward.argtypes = [dims_p, i32, vp, vp, vp, f32, vp, vp, vp, vp, sz, vp]
            lib.window_forward.restype = i32
            lib.window_backward.argtypes = [dims_p, i32] + [vp] * 6 + [f32] + [vp] * 5 + [sz, vp]
            lib.window_backward.restype = i32
            lib.window_fill.argtypes = [dims_p, i32] + [vp] * 5 + [i64, vp, vp]
            lib.window_fill.restype = i32
            lib.window_step.argtypes = [dims_p, i32] + [vp] * 4 + [f32, vp, vp, i64, vp, vp, vp]
            lib.window_step.restype = i32
            _bound = lib
    return _bound


# as in delta.py: addresses as plain integers, the raw stream query, messages only on failure
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t):
    return None if t is None else t.data_ptr()


_want = ssd._want


def _check_keys(k, v, lead):
    """Shape and type of k and v; `lead` leading axes (2: [b, L], 1: [b])."""
    ks = k.shape
    if len(ks) != lead + 2:
        raise ValueError("k and v must be [.., G, P]")
    if not k.is_cuda or not k.is_contiguous():
        raise ValueError("k must be a contiguous CUDA tensor")
    code = ssd.SSD_BF16 if k.dtype is _BF16 else ssd._dtype_code(k)
    index = k.get_device()
    _want("v", v, ks, k.dtype, index)
    return code, ks, index


def _check_queries(q, k, v, lead):
    code, ks, index = _check_keys(k, v, lead)
    qs = q.shape
    if len(qs) != lead + 2 or qs[:lead] != ks[:lead] or qs[-1] != ks[-1]:
        raise ValueError("q [.., H, P] and k, v [.., G, P] need the same leading axes and width")
    if ks[-2] < 1 or qs[-2] % ks[-2]:
        raise ValueError(f"heads ({qs[-2]}) must be a multiple of key groups ({ks[-2]})")
    _want("q", q, qs, k.dtype, index)
    return code, qs, ks[-2], index


def _check_ring(k_cache, v_cache, dtype, G, P, window, sinks, b, cache_index, index):
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache and v_cache must be [slots, sinks + window, G, P]")
    _want("k_cache", k_cache, (shape[0], sinks + window, G, P), dtype, index)
    _want("v_cache", v_cache, shape, dtype, index)
    if cache_index is not None:
        _want("cache_index", cache_index, (b,), _I32, index)
    return shape[0]


def workspace_bytes(dims: WindowDims, dtype_code: int, backward: bool) -> int:
    n = _lib().window_workspace_bytes(ctypes.byref(dims), dtype_code, int(backward))
    if n == 0:
        ssd._check(_lib().window_supported(ctypes.byref(dims), dtype_code) or 1)
    return int(n)


def _sequence(q, k, v, window, sinks, valid_len, simt):
    code, (b, L, H, P), G, index = _check_queries(q, k, v, 2)
    if valid_len is not None:
        _want("valid_len", valid_len, (b,), _I32, index)
    return code, WindowDims(b, L, H, P, G, window, sinks, WINDOW_FLAG_SIMT if simt else 0, 0), b, L, H, P, index


def window_forward(q, k, v, window, sinks=0, scale=None, valid_len=None, return_lse=True, simt=False, check_status=False):
    """Attention with a sliding window and sinks over sequences.  Returns ``(o, lse)``.

    q [b, L, H, P] and k, v [b, L, G, P] in fp32 or bf16; token t sees token s where s <= t
    and (t - s < window or s < sinks).  ``scale`` defaults to P ** -0.5; valid_len int32 [b]
    or None.  lse [b, H, L] fp32 is what :func:`window_backward` needs (None unless wanted).
    ``simt`` keeps fp32 operands in bf16 too, on CUDA cores; ``check_status`` synchronises and raises
    SsdError when valid_len entries had to be clamped.
    """
    code, dims, b, L, H, P, index = _sequence(q, k, v, window, sinks, valid_len, simt)
    o = torch.empty_like(q)
    lse = torch.empty(b, H, L, device=q.device, dtype=_F32) if return_lse else None
    ws = torch.empty(workspace_bytes(dims, code, False), dtype=torch.uint8, device=q.device)
    with ssd.on_device(index):
        ssd._check(_lib().window_forward(
            ctypes.byref(dims), code, q.data_ptr(), k.data_ptr(), v.data_ptr(), P ** -0.5 if scale is None else scale,
            _ptr(valid_len), o.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _raw_stream(index)))
    if check_status:
        ssd.workspace_status(ws)
    return o, lse


def window_backward(q, k, v, o, lse, do, window, sinks=0, scale=None, valid_len=None, simt=False, check_status=False):
    """Gradients for ``do`` at the forward's ``o`` and ``lse``: a dict with dq, dk and dv."""
    code, dims, b, L, H, P, index = _sequence(q, k, v, window, sinks, valid_len, simt)
    _want("o", o, q.shape, q.dtype, index)
    _want("do", do, q.shape, q.dtype, index)
    _want("lse", lse, (b, H, L), _F32, index)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
    ws = torch.empty(workspace_bytes(dims, code, True), dtype=torch.uint8, device=q.device)
    with ssd.on_device(index):
        ssd._check(_lib().window_backward(
            ctypes.byref(dims), code, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
            P ** -0.5 if scale is None else scale, _ptr(valid_len), out["dq"].data_ptr(), out["dk"].data_ptr(),
            out["dv"].data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(index)))
    if check_status:
        ssd.workspace_status(ws)
    return out


def window_fill(k, v, k_cache, v_cache, window, sinks=0, valid_len=None, cache_index=None):
    """Writes the tokens of prompts k, v [b, L, G, P] that later tokens see into rings
    k_cache, v_cache [slots, sinks + window, G, P]: row i's into slot cache_index[i] (int32 [b]; a slot
    outside the pool marks a row that is not kept) or slot i.  No two rows may name the same slot."""
    code, (b, L, G, P), index = _check_keys(k, v, 2)
    slots = _check_ring(k_cache, v_cache, k.dtype, G, P, window, sinks, b, cache_index, index)
    if valid_len is not None:
        _want("valid_len", valid_len, (b,), _I32, index)
    dims = WindowDims(b, L, G, P, G, window, sinks, WINDOW_FLAG_SIMT, 0)
    with ssd.on_device(index):
        ssd._check(_lib().window_fill(
            ctypes.byref(dims), code, k.data_ptr(), v.data_ptr(), _ptr(valid_len), k_cache.data_ptr(), v_cache.data_ptr(),
            slots, _ptr(cache_index), _raw_stream(index)))


def window_step(q, k, v, k_cache, v_cache, position, window, sinks=0, scale=None, cache_index=None):
    """One decoded token per request; the rings are updated in place.  Returns o.

    q [b, H, P], k, v [b, G, P] (fp32 or bf16), k_cache, v_cache [slots, sinks + window, G, P],
    position int32 [b] (the tokens before this one), cache_index int32 [b] (each request's slot; a
    slot outside the pool, or a negative position, marks an absent request, whose o is 0) or None (slot i).
    No two requests may name the same slot.
    """
    code, (b, H, P), G, index = _check_queries(q, k, v, 1)
    slots = _check_ring(k_cache, v_cache, k.dtype, G, P, window, sinks, b, cache_index, index)
    _want("position", position, (b,), _I32, index)
    dims = WindowDims(b, 1, H, P, G, window, sinks, WINDOW_FLAG_SIMT, 0)
    o = torch.empty_like(q)
    with ssd.on_device(index):
        ssd._check(_lib().window_step(
            ctypes.byref(dims), code, q.data_ptr(), k.data_ptr(), v.data_ptr(), position.data_ptr(),
            P ** -0.5 if scale is None else scale, k_cache.data_ptr(), v_cache.data_ptr(), slots, _ptr(cache_index),
            o.data_ptr(), _raw_stream(index)))
    return o
