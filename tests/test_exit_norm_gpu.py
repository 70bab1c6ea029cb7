"""GPU parity of the exit norm (norm_group_gated, include/norm.h) and of the scan's one-token step (ssd_step)
against the fp64 oracle (oracle/window.py).

Bars (normwise): fp32 outputs 2e-6 (a dozen roundings of 2^-24, exp and a division at a few units each, sums of up to
16384 terms pairwise over threads); bf16 outputs 2^-9 against the fp64 value rounded to bf16 (values near a tie may
differ, by one step of 2^-8: at fp32 noise of 2^-20 one in 2^11 of them); weight gradients 1e-5 (up to a few thousand
rows added in fp32).  The step of the scan: states 1e-6 (three roundings), y 1e-6 in fp32."""
import numpy as np
import pytest

from oracle import window as ow

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BAR = {torch.float32: 2e-6, torch.bfloat16: 2.0 ** -9}


@pytest.fixture(scope="module")
def nm():
    from state_space_model_mamba_gb300 import norm
    return norm


def rel(got, ref, floor=0.0):
    bf16 = got.dtype == torch.bfloat16
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all()
    if bf16:
        ref = torch.from_numpy(ref).bfloat16().double().numpy()
    return np.linalg.norm(got - ref) / max(np.linalg.norm(ref), floor, 1e-30)


def make(rows, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, z, dy = (torch.randn(rows, D, generator=g, device="cuda") for _ in range(3))
    x = x + 0.3 * torch.randn(1, D, generator=g, device="cuda")
    w, b = 1 + 0.1 * torch.randn(D, generator=g, device="cuda"), 0.2 * torch.randn(D, generator=g, device="cuda")
    return x.to(dtype), (2 * z).to(dtype), dy.to(dtype), w, b


def compare(nm, rows, D, groups, dtype, gate, first, center, act, bias, seed=0, eps=1e-5):
    x, z, dy, w, b = make(rows, D, dtype, rows + D + groups + seed)
    z, b = (z if gate else None), (b if bias else None)
    form = dict(bias=b, gate=z, groups=groups, eps=eps, center=center, activation=act, gate_first=first)
    y = nm.group_norm_gated(x, w, **form)
    g = nm.group_norm_gated_backward(dy, x, w, **form)

    def np64(t):
        return None if t is None else t.double().cpu().numpy()

    ry, rg = ow.group_norm(np64(x), np64(w), np64(b), np64(z), groups, eps, center, act, first, dy=np64(dy))
    # groups of one or two columns: the terms of du cancel to eps of either; dgate of a gate that comes first as well
    width = D // groups
    floor = np.linalg.norm(np64(dy)) if width <= 2 else 0.0
    bar = BAR[dtype]
    assert rel(y, ry, floor) <= bar
    wide = 1.0 if width > 2 else 300.0  # rstd up to eps^-1/2
    assert rel(g["dx"], rg["dx"], floor) <= bar * wide
    assert (g["dgate"] is None) == (z is None) and (g["dbias"] is None) == (b is None)
    if gate:
        assert rel(g["dgate"], rg["dgate"], floor) <= bar * wide
    assert rel(g["dweight"], rg["dweight"], floor) <= 1e-5
    if bias:
        assert rel(g["dbias"], rg["dbias"]) <= 1e-5


FORMS = [(gate, first, center, act, bias) for gate, first in ((False, False), (True, False), (True, True))
         for center, act, bias in ((True, "silu", True), (False, "silu", False), (True, "sigmoid", False), (False, None, True))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate,first,center,act,bias", FORMS)
def test_forms(nm, gate, first, center, act, bias, dtype):
    compare(nm, 37, 5 * 64, 5, dtype, gate, first, center, act, bias)


# every thread count and vector width: groups of 8 .. 16384 columns in 16-byte pieces, odd ones, one column
SHAPES = [(3, 32, 1), (300, 40, 5), (1, 5120, 80), (513, 5120, 80), (5, 640, 10), (4, 96, 1), (7, 768, 8), (2, 1024, 4), (3, 512, 1),
          (2, 1040, 2), (3, 2048, 1), (2, 2560, 1), (3, 4096, 1), (2, 5120, 1), (2, 8192, 1), (1, 16384, 1), (2, 16384, 2),
          (5, 7, 1), (30, 75, 25), (3, 129, 1), (3, 2 * 515, 2), (2, 1025, 1), (2, 3001, 1), (2, 5001, 1), (1, 16383, 1),
          (4, 81 * 8, 81), (2, 4096, 1024), (3, 7, 7), (2, 16381, 16381)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D,groups", SHAPES)
def test_shapes(nm, rows, D, groups, dtype):
    # one column: centred it would be noise over sqrt(eps)
    compare(nm, rows, D, groups, dtype, True, False, D > groups, "silu", True)
    if D > groups:
        compare(nm, rows, D, groups, dtype, True, True, True, "silu", False, seed=1)


def test_leading_axes_and_values_at_the_ends(nm):
    x, z, dy, w, b = make(24, 128, torch.bfloat16, 1)
    y = nm.group_norm_gated(x.view(2, 3, 4, 128), w, gate=z.view(2, 3, 4, 128), groups=2)
    assert torch.equal(y.view(24, 128), nm.group_norm_gated(x, w, gate=z, groups=2))
    # gates at the ends of the type: silu(-big) = -0, silu(big) = big, nothing becomes NaN; rows of zeros stay finite
    z[0, :] = -3e38
    z[1, :] = 300.0
    z[2, :] = -300.0
    x[3, :] = 0
    for first in (False, True):
        y = nm.group_norm_gated(x, w, gate=z, groups=2, gate_first=first)
        g = nm.group_norm_gated_backward(dy, x, w, gate=z, groups=2, gate_first=first)
        assert torch.isfinite(y.float()).all() and not y[0].any() and not y[2].any()
        assert torch.isfinite(g["dgate"][1:].float()).all() and torch.isfinite(g["dx"].float()).all()
    # a NaN stays in its group of its row
    x[5, 3] = float("nan")
    y = nm.group_norm_gated(x, w, gate=z, groups=2)
    assert torch.isnan(y[5, :64].float()).all() and torch.isfinite(y[5, 64:].float()).all()
    assert torch.isfinite(y[[0, 1, 2, 3, 4, 6]].float()).all()


def test_large_means_do_not_cancel(nm):
    """Groups whose mean is a thousand times their spread: the variance is taken about the mean."""
    x, z, dy, w, b = make(50, 256, torch.float32, 2)
    x = 1000.0 + x
    y = nm.group_norm_gated(x, w, gate=z, groups=4)
    ref = ow.group_norm(x.double().cpu().numpy(), w.double().cpu().numpy(), None, z.double().cpu().numpy(), 4, 1e-5, True, "silu", False)
    # the mean itself is off by 2^-24 of 1000 times a few roundings, of a spread of 1
    assert rel(y, ref) <= 1000 * 4 * 2.0 ** -24


def test_in_place_fixed_order_graph_and_stream(nm):
    import ctypes
    from state_space_model_mamba_gb300 import ssd
    x, z, dy, w, b = make(700, 5120, torch.bfloat16, 3)
    form = dict(bias=b, gate=z, groups=40)
    y, g = nm.group_norm_gated(x, w, **form), nm.group_norm_gated_backward(dy, x, w, **form)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, g2 = nm.group_norm_gated(x, w, **form), nm.group_norm_gated_backward(dy, x, w, **form)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, g3 = nm.group_norm_gated(x, w, **form), nm.group_norm_gated_backward(dy, x, w, **form)
    y3.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)
    for k in g:
        assert torch.equal(g[k], g2[k]) and torch.equal(g[k], g3[k])
    # y over x; dx over x and dgate over the gate
    lib, s = nm._lib(), torch.cuda.current_stream().cuda_stream
    p = [t.data_ptr() for t in (x.clone(), z.clone(), w, b)]
    xi, zi = x.clone(), z.clone()
    ssd._check(lib.norm_group_gated(1, xi.data_ptr(), z.data_ptr(), p[2], p[3], 1e-5, 1, 1, xi.data_ptr(), 700, 5120, 40, s))
    torch.cuda.synchronize()
    assert torch.equal(xi, y)
    xi = x.clone()
    ssd._check(lib.norm_group_gated_backward(1, dy.data_ptr(), xi.data_ptr(), zi.data_ptr(), p[2], p[3], 1e-5, 1, 1, xi.data_ptr(),
                                             zi.data_ptr(), None, None, 700, 5120, 40, None, 0, s))
    torch.cuda.synchronize()
    assert torch.equal(xi, g["dx"]) and torch.equal(zi, g["dgate"])


def test_offsets_past_32_bits(nm):
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    rows, D = 440000, 5120
    x = torch.randn(rows, D, device="cuda", dtype=torch.bfloat16)
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    y = nm.group_norm_gated(x, w, gate=x, groups=80)
    g = nm.group_norm_gated_backward(y, x, w, gate=x, groups=80)
    tail = x[-50:].contiguous()
    ty = nm.group_norm_gated(tail, w, gate=tail, groups=80)
    tg = nm.group_norm_gated_backward(ty, tail, w, gate=tail, groups=80)
    assert torch.equal(y[-50:], ty) and torch.equal(g["dx"][-50:], tg["dx"]) and torch.equal(g["dgate"][-50:], tg["dgate"])


def test_refusals(nm):
    x, z, dy, w, b = make(4, 64, torch.bfloat16, 4)
    for kw in (dict(groups=5), dict(groups=0), dict(activation="tanh"), dict(gate_first=True), dict(gate=z.float()), dict(gate=z[:2]),
               dict(bias=b[:32]), dict(bias=b.double())):
        with pytest.raises(ValueError):
            nm.group_norm_gated(x, w, **kw)
        with pytest.raises(ValueError):
            nm.group_norm_gated_backward(dy, x, w, **kw)
    for a, ww in ((x.half(), w), (x.t(), w), (x, w.bfloat16()), (x, w[:32])):
        with pytest.raises((ValueError, TypeError)):
            nm.group_norm_gated(a, ww)
    from state_space_model_mamba_gb300 import ssd
    with pytest.raises(ssd.SsdError, match="16384"):
        nm.group_norm_gated(torch.zeros(1, 16388, device="cuda"), torch.zeros(16388, device="cuda"))


# ------------------------------------------------------------------ the scan's step
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,H,P,N,G,slots", [(1, 80, 64, 128, 1, 4), (5, 4, 40, 16, 2, 9), (3, 6, 4, 4, 3, 3), (2, 4, 128, 256, 4, 2),
                                             (4, 2, 36, 100, 1, 8), (33, 8, 64, 64, 8, 40)])
def test_scan_step(b, H, P, N, G, slots, dtype):
    from state_space_model_mamba_gb300 import ssd
    r = np.random.default_rng(b + P + N)

    def t(a, d=torch.float32):
        return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(d)

    x, B, C = (t(r.standard_normal(s), dtype) for s in ((b, H, P), (b, G, N), (b, G, N)))
    dt, A, D = t(r.random((b, H))), t(-3 * r.random(H)), t(r.standard_normal(H))
    pool = t(r.standard_normal((slots, H, P, N)))
    index = None if slots == b else r.permutation(slots)[:b]
    if index is not None and b > 2:
        index[1] = slots if b % 2 else -1
    args = [a.double().cpu().numpy() for a in (x, dt, A, B, C, D)]
    ry, rs = ow.ssd_step(*args, pool.double().cpu().numpy(), index)
    y = ssd.ssd_step(x, dt, A, B, C, D, pool, state_index=None if index is None else torch.tensor(index, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert rel(y, ry) <= (1e-6 if dtype == torch.float32 else 2.0 ** -9)
    assert rel(pool, rs) <= 1e-6
    if index is not None and b > 2:
        assert not y[1].any()


def test_scan_steps_are_the_scan():
    """Prefill with ssd_forward, then steps from its final states, against the whole sequence."""
    import oracle
    from state_space_model_mamba_gb300 import ssd
    from state_space_model_mamba_gb300.inputs import generate_small
    i = generate_small(2, 140, 4, 64, 128, 2, seed=7, init_std=0.3, d_final_std=1.0, valid_len=None, bf16=True)
    y, _ = oracle.forward(i["x"], i["dt"], i["A"], i["B"], i["C"], i["D"], i["init"], None)

    def t(a, d=torch.float32):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(d)

    bf = torch.bfloat16
    x, B, C = (t(i[n], bf) for n in "xBC")
    dt, A, D, init = (t(i[n]) for n in ("dt", "A", "D", "init"))
    lengths = torch.tensor([130, 71], dtype=torch.int32, device="cuda")
    _, state = ssd.ssd_forward(x, dt, A, B, C, D, 128, init_state=init, valid_len=lengths)
    pool, slots = torch.zeros(5, 4, 64, 128, device="cuda"), torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    rows = torch.arange(2, device="cuda")
    for k in range(10):
        at = (lengths + k).long()
        got = ssd.ssd_step(x[rows, at], dt[rows, :, at].contiguous(), A, B[rows, at], C[rows, at], D, pool, state_index=slots)
        ref = y[np.arange(2), at.cpu().numpy()]
        # bf16 products in the chunked prefill's state (the scan's own bar is 2e-2), rounding of y
        assert np.linalg.norm(got.double().cpu().numpy() - ref) <= 2e-2 * np.linalg.norm(ref)


def test_scan_step_refusals():
    from state_space_model_mamba_gb300 import ssd
    x, dt, A, B, D = (torch.zeros(*s, device="cuda") for s in ((2, 4, 8), (2, 4), (4,), (2, 2, 8), (4,)))
    pool = torch.zeros(3, 4, 8, 8, device="cuda")
    ok = [x, dt, A, B, B, D, pool]
    ssd.ssd_step(*ok)
    for i, bad in ((0, x[0]), (0, x.bfloat16()), (1, dt[:1]), (2, A.double()), (3, B.transpose(0, 1)), (4, B[:, :1]), (6, pool[..., :4]),
                   (6, pool.bfloat16()), (6, pool[0])):
        a = list(ok)
        a[i] = bad
        with pytest.raises((ValueError, TypeError)):
            ssd.ssd_step(*a)
    with pytest.raises(ValueError):
        ssd.ssd_step(*ok, state_index=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ssd.SsdError, match="slots"):
        ssd.ssd_step(*ok[:6], pool[:1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D,groups", [(5, 128, 2), (1, 512, 4), (7, 75, 25), (3, 2048, 1)])
def test_without_eps(nm, rows, D, groups, dtype):
    """eps = 0 is harmless where no group is constant, whatever the threads that have no row make of theirs."""
    compare(nm, rows, D, groups, dtype, True, False, True, "silu", True, eps=0.0)
    compare(nm, rows, D, groups, dtype, False, False, False, "silu", True, seed=1, eps=0.0)
