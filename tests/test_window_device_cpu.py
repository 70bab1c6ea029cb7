"""Calls of window attention, the exit norm and the scan's step on tensors of a device that is not the current one (no
GPU: stand-ins, as in test_bindings_device_cpu.py)."""
import types

import pytest
import torch

from state_space_model_mamba_gb300 import norm, ssd, window
from test_bindings_device_cpu import Machine
from test_bindings_device_cpu import Tensor as Standin


class Tensor(Standin):
    def get_device(self):
        return self.device.index


@pytest.fixture
def machine(monkeypatch):
    m = Machine(monkeypatch)
    fake = ssd.torch
    fake._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: 0)
    monkeypatch.setattr(window, "torch", fake)
    monkeypatch.setattr(window, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(window, "_lib", lambda: m)
    return m


def calls(index):
    def t(*shape, dtype=torch.float32):
        return Tensor(*shape, dtype=dtype, index=index)

    q, k = t(2, 8, 4, 16), t(2, 8, 2, 16)
    ring, one = [t(3, 7, 2, 16), t(3, 7, 2, 16)], [t(2, 4, 16), t(2, 2, 16), t(2, 2, 16)]
    x, w = t(3, 64), t(64)
    return {
        "window_forward": lambda: window.window_forward(q, k, k, 5, 2, check_status=True),
        "window_backward": lambda: window.window_backward(q, k, k, q, t(2, 4, 8), q, 5, 2, check_status=True),
        "window_fill": lambda: window.window_fill(k, k, *ring, 5, 2),
        "window_step": lambda: window.window_step(*one, *ring, t(2, dtype=torch.int32), 5, 2),
        "norm_group_gated": lambda: norm.group_norm_gated(x, w, w, x, groups=4),
        "norm_group_gated_backward": lambda: norm.group_norm_gated_backward(x, x, w, w, x, groups=4),
        "ssd_step": lambda: ssd.ssd_step(t(2, 4, 8), t(2, 4), t(4), t(2, 2, 16), t(2, 2, 16), t(4), t(3, 4, 8, 16)),
    }


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_launches_find_the_tensors_device(machine, name):
    calls(1)[name]()
    assert name in [n for n, _ in machine.launches] and all(at == 1 for _, at in machine.launches), machine.launches
    assert machine.now == 0


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_the_current_device_is_not_switched(machine, name):
    calls(0)[name]()
    assert name in [n for n, _ in machine.launches] and machine.switches == 0
