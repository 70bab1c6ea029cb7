"""Host-side checks of include/window.h, the exit norm in include/norm.h and ssd_step (no GPU): exports, workspace
sizes, and refusals before anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

from state_space_model_mamba_gb300 import build as ssd_build
from state_space_model_mamba_gb300 import norm, ssd, window

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUF = ctypes.c_void_p(1 << 20)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    norm._lib()
    return window._lib()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "window.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(window_[a-z0-9_]+)\s*\(", text))
    assert names == set(window.EXPORTED)
    for n in names:
        assert hasattr(lib, n)
    assert "ssd_step" in ssd.EXPORTED and hasattr(lib, "ssd_step")


def dims(**kw):
    d = dict(batch=2, seqlen=100, nheads=4, headdim=64, ngroups=2, window=16, sinks=4, flags=0, reserved=0)
    d.update(kw)
    return ctypes.byref(window.WindowDims(*d.values()))


@pytest.mark.parametrize("kw,code,status", [
    ({}, 0, 0), ({}, 1, 0), (dict(flags=1), 1, 0), (dict(headdim=4), 0, 0), (dict(headdim=12, flags=1), 1, 0),
    (dict(sinks=0), 1, 0), (dict(window=1), 1, 0), (dict(window=1 << 20, sinks=1 << 20), 1, 0), (dict(nheads=256, ngroups=1), 1, 0),
    (dict(batch=0), 0, 1), (dict(seqlen=0), 0, 1), (dict(seqlen=-1), 1, 1), (dict(ngroups=0), 0, 1), (dict(ngroups=3), 0, 1),
    (dict(window=0), 1, 1), (dict(window=-4), 1, 1), (dict(sinks=-1), 1, 1), (dict(reserved=1), 0, 1), (dict(flags=2), 1, 1),
    ({}, 2, 1), (dict(headdim=132), 0, 2), (dict(headdim=6), 0, 2), (dict(headdim=12), 1, 2), (dict(headdim=136), 1, 2),
    (dict(seqlen=1 << 40), 0, 2), (dict(batch=1 << 40), 0, 2), (dict(window=1 << 40), 1, 2), (dict(sinks=1 << 40), 1, 2),
])
def test_supported(lib, kw, code, status):
    assert lib.window_supported(dims(**kw), code) == status
    for backward in (0, 1):
        assert (lib.window_workspace_bytes(dims(**kw), code, backward) > 0) == (status == 0)
    assert bool(lib.ssd_last_error()) == (status != 0)


def test_window_calls_reject_bad_arguments_before_launch(lib):
    d, big = dims(), 1 << 40
    fwd = [BUF, BUF, BUF, 1.0, None, BUF, None, BUF, big, None]
    for i in (0, 1, 2, 5, 7):
        for bad in (None, ODD):
            a = list(fwd)
            a[i] = bad
            assert lib.window_forward(d, 1, *a) == ssd.SSD_ERR_INVALID_ARG
    assert lib.window_forward(d, 1, *(fwd[:6] + [ODD] + fwd[7:])) == ssd.SSD_ERR_INVALID_ARG
    assert lib.window_forward(d, 1, *(fwd[:8] + [16, None])) == ssd.SSD_ERR_WORKSPACE
    bwd = [BUF] * 6 + [1.0, None] + [BUF] * 4 + [big, None]
    for i in (0, 1, 2, 3, 4, 5, 8, 9, 10, 11):
        a = list(bwd)
        a[i] = None
        assert lib.window_backward(d, 1, *a) == ssd.SSD_ERR_INVALID_ARG
        assert b"NULL" in lib.ssd_last_error()
    assert lib.window_backward(d, 1, *(bwd[:12] + [1 << 10, None])) == ssd.SSD_ERR_WORKSPACE
    fill = [BUF, BUF, None, BUF, BUF, 2, None, None]
    for i, bad in ((0, None), (1, ODD), (3, None), (4, ODD), (5, 0), (5, 1), (5, 1 << 40)):
        a = list(fill)
        a[i] = bad
        assert lib.window_fill(d, 1, *a) == ssd.SSD_ERR_INVALID_ARG
    one = dims(seqlen=1)
    step = [BUF, BUF, BUF, BUF, 1.0, BUF, BUF, 2, None, BUF, None]
    assert lib.window_step(d, 1, *step) == ssd.SSD_ERR_INVALID_ARG  # 100 tokens
    for i, bad in ((0, None), (1, None), (2, ODD), (3, None), (5, None), (6, ODD), (7, 0), (7, 1), (9, None)):
        a = list(step)
        a[i] = bad
        assert lib.window_step(one, 1, *a) == ssd.SSD_ERR_INVALID_ARG, (i, bad)
    assert lib.window_step(dims(seqlen=1, window=0), 1, *step) == ssd.SSD_ERR_INVALID_ARG


def test_exit_norm_rejects_bad_arguments_before_launch(lib):
    ok = [BUF, BUF, BUF, None, 1e-5, 1, 1, BUF, 4, 64, 4, None]
    for i, bad, status in ((0, None, 1), (1, ODD, 1), (2, None, 1), (3, ODD, 1), (5, 3, 1), (5, -1, 1), (6, 4, 1), (7, None, 1),
                           (8, 0, 1), (9, 0, 1), (10, 0, 1), (10, 5, 1), (9, 16388, 2), (8, 1 << 31, 2)):
        a = list(ok)
        a[i] = bad
        assert lib.norm_group_gated(1, *a) == status, (i, bad)
    assert lib.norm_group_gated(3, *ok) == 1
    assert lib.norm_group_gated(1, *([BUF, None] + ok[2:6] + [2] + ok[7:])) == 1  # gate first without a gate
    bw = [BUF, BUF, BUF, BUF, None, 1e-5, 1, 1, BUF, BUF, BUF, None, 4, 64, 4, BUF, 1 << 30, None]
    for i, bad in ((0, None), (1, None), (3, None), (8, ODD), (9, None), (2, None), (15, None)):
        a = list(bw)
        a[i] = bad
        assert lib.norm_group_gated_backward(1, *a) == 1, (i, bad)
    assert lib.norm_group_gated_backward(1, *(bw[:16] + [64, None])) == ssd.SSD_ERR_WORKSPACE
    assert lib.norm_group_workspace_bytes(1, 4, 64, 4) >= 2 * 4 * 64 and lib.norm_group_workspace_bytes(1, 4, 64, 5) == 0


def test_scan_step_rejects_bad_arguments_before_launch(lib):
    def sd(**kw):
        d = dict(batch=2, seqlen=1, nheads=4, headdim=64, dstate=128, ngroups=2, chunk_len=64, flags=0, reserved=0)
        d.update(kw)
        return ctypes.byref(ssd.SsdDims(*d.values()))

    step = [BUF] * 7 + [2, None, BUF, None]
    assert lib.ssd_step(sd(seqlen=2), 1, *step) == 1
    for i in (0, 1, 2, 3, 4, 5, 6, 9):
        for bad in (None, ODD):
            a = list(step)
            a[i] = bad
            assert lib.ssd_step(sd(), 1, *a) == 1
    for slots in (0, 1, 1 << 40):
        assert lib.ssd_step(sd(), 1, *(step[:7] + [slots] + step[8:])) == 1
    assert lib.ssd_step(sd(headdim=6), 1, *step) == 2 and lib.ssd_step(sd(dstate=260), 1, *step) == 2
    assert lib.ssd_step(sd(batch=1 << 28), 1, *(step[:8] + [BUF] + step[9:])) == 2


def test_bindings_refuse_wrong_tensors(lib):
    q, k = torch.zeros(1, 4, 4, 8), torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        window.window_forward(q, k, k, 4)
    with pytest.raises(ValueError, match="CUDA"):
        norm.group_norm_gated(torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_step(torch.zeros(1, 4, 8), torch.zeros(1, 4), torch.zeros(4), torch.zeros(1, 2, 8), torch.zeros(1, 2, 8),
                     torch.zeros(4), torch.zeros(1, 4, 8, 8))


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_scales_that_are_not_finite_are_refused(lib, scale):
    big = 1 << 40
    assert lib.window_forward(dims(), 1, BUF, BUF, BUF, scale, None, BUF, None, BUF, big, None) == ssd.SSD_ERR_INVALID_ARG
    assert b"finite" in lib.ssd_last_error()
    assert lib.window_backward(dims(), 1, *([BUF] * 6 + [scale, None] + [BUF] * 4 + [big, None])) == ssd.SSD_ERR_INVALID_ARG
    assert lib.window_step(dims(seqlen=1), 1, BUF, BUF, BUF, BUF, scale, BUF, BUF, 2, None, BUF, None) == ssd.SSD_ERR_INVALID_ARG


def test_the_workspace_of_many_sinks_is_bounded(lib):
    """Half the tokens as sinks: the shares of their gradients stay below 2048 tiles of 128 x headdim pairs of fp32 a group;
    where everybody is seen nothing is kept at all."""
    L, groups = 131072, 2 * 2
    delta = 4 * 2 * 4 * L

    def size(**kw):
        return lib.window_workspace_bytes(dims(seqlen=L, **kw), 1, 1)

    for window_, sinks in ((1024, 4), (1024, 200), (1, 40000), (1024, L // 2), (3000, L - 4000)):
        assert delta < size(window=window_, sinks=sinks) <= delta + 2048 + groups * 2048 * 2 * 128 * 64 * 4
    none = size(window=1024, sinks=0)
    assert none <= delta + 2048
    assert size(window=1024, sinks=L) == size(window=1, sinks=L - 1) == size(window=L, sinks=4) == none
