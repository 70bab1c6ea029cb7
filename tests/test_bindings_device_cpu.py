"""Calls on tensors of a device that is not the current one (no GPU: the device query, the library and the tensors
are stand-ins): every launch of the bindings happens with the tensors' device made current, and no device is
switched where it already is."""
import contextlib
import types

import pytest
import torch

from state_space_model_mamba_gb300 import delta, mamba3, norm, ssd


class Tensor:
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, index=1):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096


class Machine:
    """Two devices, 0 the current one; records the device that each launch finds."""

    def __init__(self, monkeypatch):
        self.now, self.switches, self.launches = 0, 0, []

        @contextlib.contextmanager
        def device(index):
            self.now, before = index, self.now
            self.switches += 1
            yield
            self.now = before

        def like(t, **_):
            return Tensor(*t.shape, dtype=t.dtype, index=t.device.index)

        def empty(*shape, device=None, dtype=torch.float32):
            shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
            return Tensor(*shape, dtype=dtype, index=device.index)

        fake = types.SimpleNamespace(empty=empty, empty_like=like, cuda=types.SimpleNamespace(device=device),
                                     **{n: getattr(torch, n) for n in ("float32", "bfloat16", "uint8", "int32", "int64",
                                                                       "float8_e4m3fn")})
        for m in (ssd, delta, norm, mamba3):
            monkeypatch.setattr(m, "torch", fake)
        monkeypatch.setattr(ssd, "_get_device", lambda: self.now, raising=False)
        monkeypatch.setattr(ssd, "load_library", lambda: self)
        monkeypatch.setattr(ssd, "_stream_ptr", lambda d: None)
        monkeypatch.setattr(mamba3, "_stream", lambda d: None)
        for m in (delta, norm):
            monkeypatch.setattr(m, "_raw_stream", lambda index: 0)
        for m in (delta, norm, mamba3):
            monkeypatch.setattr(m, "_lib", lambda: self)

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 64
            if not name.endswith("_supported"):
                self.launches.append((name, self.now))
            return 0
        return call


def calls(index):
    def t(*shape, dtype=torch.float32):
        return Tensor(*shape, dtype=dtype, index=index)

    seq = [t(2, 8, 2, 16), t(2, 8, 2, 16), t(2, 8, 4, 8), t(2, 4, 8), t(2, 4, 8)]
    one = [t(2, 2, 16), t(2, 2, 16), t(2, 4, 8), t(2, 4), t(2, 4)]
    scan = [t(2, 8, 4, 8), t(2, 4, 8), t(4), t(2, 8, 2, 16), t(2, 8, 2, 16), t(4)]
    x, w = t(3, 64), t(64)
    y = [t(3, 1, 4, 8), t(3, 1, 4, 16), t(3, 1, 4, 16), t(3, 4)]
    quat = t(2, 8, 4, 2, 4)
    return {
        "delta_forward": lambda: delta.delta_forward(*seq, check_status=True),
        "delta_backward": lambda: delta.delta_backward(*seq, t(2, 8, 4, 8)),
        "delta_step": lambda: delta.delta_step(*one, t(5, 4, 8, 16)),
        "norm_add_rms": lambda: norm.add_rms_norm(x, w),
        "norm_add_rms_fp8": lambda: norm.add_rms_norm_fp8(x, w, group=32),
        "norm_add_rms_backward": lambda: norm.add_rms_norm_backward(x, x, w),
        "ssd_forward": lambda: ssd.ssd_forward(*scan, 64, check_status=True),
        "ssd_backward": lambda: ssd.ssd_backward(*scan, 64, t(2, 8, 4, 8)),
        "ssd_state_moments": lambda: ssd.state_moments(scan[0], scan[1], scan[2], scan[3]),
        "ssd_state_pr": lambda: ssd.state_pr(t(2, 4, 16, 16), t(2, 4, 16), t(2)),
        "ssd_workspace_status": lambda: ssd.workspace_status(t(64, dtype=torch.uint8)),
        "ssd_wait_selftest": lambda: ssd.wait_selftest(t(64, dtype=torch.uint8), 1, True),
        "m3_quat_cumprod": lambda: mamba3.quat_cumprod(quat),
        "m3_quat_cumprod_backward": lambda: mamba3.quat_cumprod_backward(quat, None, quat),
        "m3_y_diag": lambda: mamba3.y_diag(*y),
        "m3_y_diag_backward": lambda: mamba3.y_diag_backward(t(3, 1, 4, 8), *y),
    }


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_launches_find_the_tensors_device(monkeypatch, name):
    m = Machine(monkeypatch)
    calls(1)[name]()
    assert name in [n for n, _ in m.launches] and all(at == 1 for _, at in m.launches), m.launches
    assert m.now == 0


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_the_current_device_is_not_switched(monkeypatch, name):
    m = Machine(monkeypatch)
    calls(0)[name]()
    assert name in [n for n, _ in m.launches] and m.switches == 0
