"""Thin Python binding of the gated delta rule's entry points of ``libssd.so``
(``include/delta.h``): the chunked forward and its recompute backward, and the
one-token step over a pool of states.

Argument marshalling only, as :mod:`ssd`: torch CUDA tensors supply memory and
streams, every step runs in the library's kernels, and a missing library or a
failed call raises.  Tensors are used on the current stream of their device.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import ssd

EXPORTED = ("delta_supported", "delta_workspace_bytes", "delta_forward", "delta_backward", "delta_step")
DELTA_FLAG_SIMT = 1

_lock = threading.Lock()
_bound = None


class DeltaDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


def _lib():
    global _bound
    if _bound is not None:
        return _bound
    with _lock:
        if _bound is None:
            lib = ssd.load_library()
            vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
            dims_p = ctypes.POINTER(DeltaDims)
            lib.delta_supported.argtypes = [dims_p, i32]
            lib.delta_supported.restype = i32
            lib.delta_workspace_bytes.argtypes = [dims_p, i32, i32]
            lib.delta_workspace_bytes.restype = sz
            lib.delta_forward.argtypes = [dims_p, i32] + [vp] * 5 + [f32] + [vp] * 4 + [vp, sz, vp]
            lib.delta_forward.restype = i32
            lib.delta_backward.argtypes = [dims_p, i32] + [vp] * 5 + [f32] + [vp] * 10 + [vp, sz, vp]
            lib.delta_backward.restype = i32
            lib.delta_step.argtypes = [dims_p, i32] + [vp] * 5 + [f32, vp, ctypes.c_int64] + [vp] * 3
            lib.delta_step.restype = i32
            _bound = lib
    return _bound


# One decoded token is a few microseconds of GPU work, so the calls below keep the host's
# part short: addresses go to ctypes as plain integers, the stream comes from the raw
# query, and what a check would print is only formed when it fails.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _want(name, t, shape, dtype, device):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on {device}")


def _check_tokens(q, k, v, g, beta, lead):
    """Shapes and types of the per-token tensors; `lead` leading axes (2: [b, L], 1: [b])."""
    vs, qs = v.shape, q.shape
    if len(vs) != lead + 2 or len(qs) != lead + 2:
        raise ValueError("q, k [.., G, N] and v [.., H, P] need the same leading axes")
    if not v.is_cuda or not v.is_contiguous():
        raise ValueError("v must be a contiguous CUDA tensor")
    dtype, device = v.dtype, v.device
    code = ssd.SSD_BF16 if dtype is _BF16 else ssd._dtype_code(v)
    G, N = qs[-2:]
    H, P = vs[-2:]
    if G < 1 or H % G:
        raise ValueError(f"heads ({H}) must be a multiple of key groups ({G})")
    gate = (vs[0], H) if lead == 1 else (vs[0], H, vs[1])
    if not (q.dtype is dtype and k.dtype is dtype and g.dtype is _F32 and beta.dtype is _F32
            and qs[:lead] == vs[:lead] and k.shape == qs and g.shape == gate and beta.shape == gate
            and q.device == device and k.device == device and g.device == device and beta.device == device
            and q.is_contiguous() and k.is_contiguous() and g.is_contiguous() and beta.is_contiguous()):
        keys = vs[:lead] + (G, N)
        _want("q", q, keys, dtype, device)
        _want("k", k, keys, dtype, device)
        _want("g", g, gate, _F32, device)
        _want("beta", beta, gate, _F32, device)
    return code, G, N, H, P


def _dims(b, L, H, P, N, G, simt=False):
    return DeltaDims(b, L, H, P, N, G, DELTA_FLAG_SIMT if simt else 0, 0)


def workspace_bytes(dims: DeltaDims, dtype_code: int, backward: bool) -> int:
    n = _lib().delta_workspace_bytes(ctypes.byref(dims), dtype_code, int(backward))
    if n == 0:
        ssd._check(_lib().delta_supported(ctypes.byref(dims), dtype_code) or 1)
    return int(n)


def _check_sequence(v, N, init_state, valid_len):
    b, _, H, P = v.shape
    if init_state is not None:
        _want("init_state", init_state, (b, H, P, N), _F32, v.device)
    if valid_len is not None:
        _want("valid_len", valid_len, (b,), _I32, v.device)


def delta_forward(q, k, v, g, beta, scale=None, init_state=None, valid_len=None, return_final_state=True,
                  simt=False, check_status=False):
    """The gated delta rule over sequences.  Returns ``(o, final_state)``.

    q, k [b, L, G, N] and v [b, L, H, P] in fp32 or bf16, g (log decay) and beta
    [b, H, L] fp32, init_state [b, H, P, N] fp32 or None, valid_len int32 [b] or
    None.  ``scale`` defaults to N ** -0.5.  ``simt`` takes the token-by-token
    kernels in bf16 too (fp32 operands throughout: fp32 outputs 1e-7 to 3e-7 off, where the
    chunked kernels' are 2e-7 to 5e-6); ``check_status`` synchronises and raises SsdError when
    valid_len entries had to be clamped.
    """
    code, G, N, H, P = _check_tokens(q, k, v, g, beta, 2)
    _check_sequence(v, N, init_state, valid_len)
    b, L = v.shape[:2]
    dims = _dims(b, L, H, P, N, G, simt)
    o = torch.empty_like(v)
    fin = torch.empty(b, H, P, N, device=v.device, dtype=_F32) if return_final_state else None
    ws = torch.empty(workspace_bytes(dims, code, False), dtype=torch.uint8, device=v.device)
    index = v.device.index
    with ssd.on_device(index):
        ssd._check(_lib().delta_forward(
            ctypes.byref(dims), code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            N ** -0.5 if scale is None else scale, _ptr(init_state), _ptr(valid_len), o.data_ptr(), _ptr(fin), ws.data_ptr(),
            ws.numel(), _raw_stream(index)))
    if check_status:
        ssd.workspace_status(ws)
    return o, fin


def delta_backward(q, k, v, g, beta, do, scale=None, d_final_state=None, init_state=None, valid_len=None,
                   want_d_init=True, simt=False, check_status=False):
    """Recompute backward for the gradient ``do`` of o (and ``d_final_state``).
    Returns a dict with dq, dk, dv, dg, dbeta and d_init (None unless wanted)."""
    code, G, N, H, P = _check_tokens(q, k, v, g, beta, 2)
    _check_sequence(v, N, init_state, valid_len)
    b, L = v.shape[:2]
    _want("do", do, v.shape, v.dtype, v.device)
    if d_final_state is not None:
        _want("d_final_state", d_final_state, (b, H, P, N), _F32, v.device)
    dims = _dims(b, L, H, P, N, G, simt)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v), dg=torch.empty_like(g),
               dbeta=torch.empty_like(beta),
               d_init=torch.empty(b, H, P, N, device=v.device, dtype=_F32) if want_d_init else None)
    ws = torch.empty(workspace_bytes(dims, code, True), dtype=torch.uint8, device=v.device)
    index = v.device.index
    with ssd.on_device(index):
        ssd._check(_lib().delta_backward(
            ctypes.byref(dims), code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            N ** -0.5 if scale is None else scale, _ptr(init_state), _ptr(valid_len), _ptr(do), _ptr(d_final_state),
            _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["d_init"]),
            _ptr(ws), ws.numel(), _raw_stream(index)))
    if check_status:
        ssd.workspace_status(ws)
    return out


def delta_step(q, k, v, g, beta, state, scale=None, state_index=None):
    """One decoded token per request; ``state`` is updated in place.  Returns o.

    q, k [b, G, N], v [b, H, P] (fp32 or bf16), g, beta [b, H] fp32, state
    [slots, H, P, N] fp32, state_index int32 [b] (each request's slot; a slot
    outside the pool marks an absent request, whose o is 0) or None (slot i).
    No two requests may name the same slot.
    """
    code, G, N, H, P = _check_tokens(q, k, v, g, beta, 1)
    b = v.shape[0]
    if state.dim() != 4:
        raise ValueError("state must be [slots, H, P, N]")
    _want("state", state, (state.shape[0], H, P, N), _F32, v.device)
    if state_index is not None:
        _want("state_index", state_index, (b,), _I32, v.device)
    dims = _dims(b, 1, H, P, N, G)
    o = torch.empty_like(v)
    index = v.device.index
    with ssd.on_device(index):
        ssd._check(_lib().delta_step(
            ctypes.byref(dims), code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            N ** -0.5 if scale is None else scale, state.data_ptr(), state.shape[0], _ptr(state_index), o.data_ptr(),
            _raw_stream(index)))
    return o
