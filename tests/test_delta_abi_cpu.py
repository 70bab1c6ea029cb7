"""Host-side checks of include/delta.h and include/norm.h (no GPU): exports,
workspace sizes, and refusals before anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

from state_space_model_mamba_gb300 import build as ssd_build
from state_space_model_mamba_gb300 import delta, norm, ssd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUF = ctypes.c_void_p(1 << 20)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    delta._lib()
    return norm._lib()


def test_every_declared_symbol_is_exported(lib):
    for header, mod in (("delta.h", delta), ("norm.h", norm)):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        names = set(re.findall(r"\b((?:delta|norm)_[a-z0-9_]+)\s*\(", text))
        assert names == set(mod.EXPORTED)
        for n in names:
            assert hasattr(lib, n)


def dims(**kw):
    d = dict(batch=2, seqlen=100, nheads=4, headdim=64, dstate=128, ngroups=2, flags=0, reserved=0)
    d.update(kw)
    return ctypes.byref(delta.DeltaDims(*d.values()))


@pytest.mark.parametrize("kw,code,status", [
    ({}, 0, 0), ({}, 1, 0), (dict(flags=1), 1, 0),
    (dict(headdim=4, dstate=256), 0, 0),
    (dict(batch=0), 0, 1), (dict(seqlen=0), 0, 1), (dict(seqlen=-1), 1, 1), (dict(ngroups=0), 0, 1),
    (dict(ngroups=3), 0, 1), (dict(reserved=1), 0, 1), (dict(flags=2), 1, 1), ({}, 2, 1),
    (dict(headdim=132), 0, 2), (dict(headdim=6), 0, 2), (dict(dstate=260), 0, 2), (dict(dstate=2), 0, 2),
    (dict(seqlen=1 << 40), 0, 2), (dict(batch=1 << 40), 0, 2),
])
def test_supported(lib, kw, code, status):
    assert lib.delta_supported(dims(**kw), code) == status
    assert (lib.delta_workspace_bytes(dims(**kw), code, 0) > 0) == (status == 0)
    assert (lib.delta_workspace_bytes(dims(**kw), code, 1) > 0) == (status == 0)
    assert bool(lib.ssd_last_error()) == (status != 0)


def test_delta_calls_reject_bad_arguments_before_launch(lib):
    d, big = dims(), 1 << 40
    fwd = [BUF] * 5 + [1.0, None, None, BUF, None, BUF, big, None]
    for i in (0, 1, 2, 3, 4, 8, 10):
        for bad in (None, ODD):
            a = list(fwd)
            a[i] = bad
            assert lib.delta_forward(d, 1, *a) == ssd.SSD_ERR_INVALID_ARG
    assert lib.delta_forward(d, 1, *(fwd[:6] + [ODD] + fwd[7:])) == ssd.SSD_ERR_INVALID_ARG
    assert lib.delta_forward(d, 1, *(fwd[:11] + [16, None])) == ssd.SSD_ERR_WORKSPACE
    bwd = [BUF] * 5 + [1.0, None, None, BUF, None] + [BUF] * 5 + [None, BUF, big, None]
    for i in (0, 1, 2, 3, 4, 8, 10, 11, 12, 13, 14, 16):
        a = list(bwd)
        a[i] = None
        assert lib.delta_backward(d, 1, *a) == ssd.SSD_ERR_INVALID_ARG
        assert b"NULL" in lib.ssd_last_error()
    assert lib.delta_backward(d, 1, *(bwd[:17] + [1 << 10, None])) == ssd.SSD_ERR_WORKSPACE
    step = [BUF] * 5 + [1.0, BUF, 2, None, BUF, None]
    assert lib.delta_step(d, 1, *step) == ssd.SSD_ERR_INVALID_ARG      # 100 tokens
    assert lib.delta_step(dims(seqlen=1), 1, *(step[:7] + [1] + step[8:])) == ssd.SSD_ERR_INVALID_ARG  # one slot for two
    assert lib.delta_step(dims(seqlen=1), 1, *(step[:7] + [0] + step[8:])) == ssd.SSD_ERR_INVALID_ARG
    assert lib.delta_step(dims(seqlen=1), 1, *(step[:6] + [None] + step[7:])) == ssd.SSD_ERR_INVALID_ARG


def test_norm_calls_reject_bad_arguments_before_launch(lib):
    ok = [BUF, None, BUF, 1e-5, BUF, None, 4, 64, None]
    for i, bad, status in ((0, None, 1), (2, None, 1), (4, ODD, 1), (1, BUF, 1), (6, 0, 1), (7, 0, 1), (7, 16385, 2),
                           (6, 1 << 31, 2)):
        a = list(ok)
        a[i] = bad
        assert lib.norm_add_rms(1, *a) == status, (i, bad)
    assert lib.norm_add_rms(3, *ok) == 1
    f8 = [BUF, None, BUF, 1e-5, BUF, BUF, None, 4, 96, 0, None]
    for group, status in ((64, 2), (16, 2), (-1, 2), (96, 2)):
        assert lib.norm_add_rms_fp8(1, *(f8[:9] + [group, None])) == status
    assert lib.norm_add_rms_fp8(1, *(f8[:5] + [None] + f8[6:])) == 1
    bw = [BUF, BUF, BUF, 1e-5, None, BUF, BUF, 4, 64, BUF, 4 * 64 * 4, None]
    assert lib.norm_backward_workspace_bytes(4, 64) == 4 * 64 * 4
    assert lib.norm_backward_workspace_bytes(4, 0) == 0
    assert lib.norm_add_rms_backward(1, *(bw[:10] + [1023, None])) == ssd.SSD_ERR_WORKSPACE
    assert lib.norm_add_rms_backward(1, *([None] + bw[1:])) == 1


def test_bindings_refuse_wrong_tensors(lib):
    b, L, G, N, H, P = 1, 4, 2, 8, 4, 8
    ok = dict(q=torch.zeros(b, L, G, N), k=torch.zeros(b, L, G, N), v=torch.zeros(b, L, H, P), g=torch.zeros(b, H, L),
              beta=torch.zeros(b, H, L))
    with pytest.raises(ValueError, match="CUDA"):
        delta.delta_forward(**ok)
    with pytest.raises(ValueError, match="CUDA"):
        norm.add_rms_norm(torch.zeros(2, 8), torch.ones(8))


def test_norm_kernels_are_those_that_some_row_takes(lib):
    """Every variant that the library holds is reached by a row of 1 .. 16384 columns, and every one reached is there."""
    import shutil
    import subprocess
    if shutil.which("nm") is None:
        pytest.skip("needs nm")
    names = subprocess.run(["nm", "-C", ssd.LIB_PATH], capture_output=True, text=True, check=True).stdout
    held = {(m[1], m[2]) + tuple(int(x) for x in m[3].split(", "))
            for m in re.finditer(r"\b(add_rms|rms_bwd)_kernel<(float|__nv_bfloat16), (\d+, \d+, \d+)[,>]", names)}
    reached = set()
    for t, wide in (("float", 4), ("__nv_bfloat16", 8)):
        for D in range(1, 16385):
            vec = wide if D % wide == 0 else 2 - D % 2
            n = D // vec
            if vec == wide:
                if n <= 32:
                    tpr, nv = 32, 1
                else:
                    tpr = next((x for x in (32, 64, 128, 160, 256, 320, 512, 1024) if n <= 2 * x), 1024)
                    nv = 2 if n <= 2048 else 4
            else:
                tpr = next((x for x in (128, 256, 512, 1024) if n <= 4 * x), 1024)
                nv = 4 if n <= 4096 else (8 if n <= 8192 else 16)
            reached |= {("add_rms", t, vec, tpr, nv), ("rms_bwd", t, vec, tpr, nv)}
    assert held == reached, (sorted(held - reached), sorted(reached - held))
