"""GPU parity of the entry norm (include/norm.h) against fp64.

Bars (normwise): fp32 outputs 1e-6 (a few roundings of 2^-24 and sums of up to
16384 terms in fp32, pairwise over threads); bf16 outputs 2^-9 against the fp64
value rounded to bf16 (only values within fp32 noise of a tie may differ); dweight 1e-5 (up to a few thousand rows added in fp32)."""
import numpy as np
import pytest

from oracle import delta as od

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BAR = {torch.float32: 1e-6, torch.bfloat16: 2.0 ** -9}


@pytest.fixture(scope="module")
def nm():
    from state_space_model_mamba_gb300 import norm
    return norm


def rel(got, ref):
    bf16 = got.dtype == torch.bfloat16
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all()
    if bf16:
        ref = torch.from_numpy(ref).bfloat16().double().numpy()
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


def make(rows, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r, dy, ds = (torch.randn(rows, D, generator=g, device="cuda").to(dtype) for _ in range(4))
    return x, r, dy, ds, 1 + 0.1 * torch.randn(D, generator=g, device="cuda")


# every thread count and vector width: multiples of 8, even, odd; one column; the largest row
SHAPES = [(1, 8), (5, 1), (3, 7), (4, 250), (2, 256), (130, 264), (3, 1000), (7, 1026), (2, 2051), (300, 2560), (2, 3000),
          (3, 4096), (2, 4100), (2, 5121), (2, 8192), (2, 10008), (1, 16384), (1, 16383), (1, 16382)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_forward_backward(nm, rows, D, dtype):
    x, r, dy, ds, w = make(rows, D, dtype, rows + D)
    y, stream = nm.add_rms_norm(x, w, 1e-5, residual=r)
    assert torch.equal(stream, (x.float() + r.float()).to(dtype))
    h = stream.double().cpu().numpy()
    assert rel(y, od.add_rms_norm(h, w.double().cpu().numpy(), 1e-5)) <= BAR[dtype]
    y0, s0 = nm.add_rms_norm(stream, w, 1e-5)
    assert s0 is stream and torch.equal(y0, y)
    for d_stream in (None, ds):
        dx, dw = nm.add_rms_norm_backward(dy, stream, w, 1e-5, d_stream=d_stream)
        rx, rw = od.add_rms_norm_backward(dy.double().cpu().numpy(), h, w.double().cpu().numpy(), 1e-5,
                                          None if d_stream is None else ds.double().cpu().numpy())
        # one column: y = sign(h) w up to eps, the two terms of dx cancel to ~eps of either
        bar = BAR[dtype] if D > 1 or d_stream is not None else 1.0
        assert rel(dx, rx) <= bar
        assert rel(dw, rw) <= 1e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D,group", [(3, 128, 0), (5, 256, 32), (4, 2560, 128), (300, 2560, 64), (2, 96, 32), (3, 250, 0),
                                          (2, 2051, 0), (1, 16384, 128), (7, 10240, 0), (129, 512, 128), (1, 1, 0)])
def test_fp8(nm, rows, D, group, dtype):
    x, r, _, _, w = make(rows, D, dtype, rows + D + group)
    y8, scales, stream = nm.add_rms_norm_fp8(x, w, 1e-5, residual=r, group=group)
    assert y8.dtype == torch.float8_e4m3fn and y8.shape == x.shape and scales.shape == (rows, D // group if group else 1)
    assert torch.equal(stream, (x.float() + r.float()).to(dtype))
    y = od.add_rms_norm(stream.double().cpu().numpy(), w.double().cpu().numpy(), 1e-5).reshape(rows, scales.shape[1], -1)
    ref = np.abs(y).max(-1) / 448.0
    assert rel(scales, ref) <= 1e-6
    q = y8.float().double().cpu().numpy().reshape(y.shape)
    # nearest e4m3: half a step of 2^-3 of the value's power of two, at least half of 2^-9; fp32 noise on ties
    err = np.abs(q - y / ref[..., None])
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y / ref[..., None]), 2.0 ** -6))) - 3)
    assert np.all(err <= 0.5 * step * (1 + 1e-4)) and np.abs(q).max() <= 448


def test_zero_rows_and_non_finite_rows(nm):
    x, r, _, _, w = make(6, 512, torch.bfloat16, 1)
    x[1] = 0
    r[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4, :128] = 0
    r[4, :128] = 0
    for group in (0, 128):
        y8, s, _ = nm.add_rms_norm_fp8(x, w, 1e-5, residual=r, group=group)
        assert torch.all(y8[1].float() == 0) and torch.all(s[1] == 0)
        assert torch.isnan(y8[2].float()).all() and torch.isnan(s[2]).all()
        assert torch.isnan(y8[3].float()[7])
        assert torch.all(y8[4, :128].float() == 0) and torch.isfinite(y8[4].float()).all()
        assert torch.isfinite(y8[[0, 4, 5]].float()).all() and torch.isfinite(s[[0, 4, 5]]).all()
    y, _ = nm.add_rms_norm(x, w, 1e-5, residual=r)
    assert torch.all(y[1] == 0) and torch.isnan(y[2]).all() and torch.isnan(y[3, 7])
    assert torch.isfinite(y[[0, 1, 4, 5]]).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("top", [1e-38, 1e-44, 2e38])
def test_fp8_scales_at_the_ends_of_fp32(nm, group, top):
    """Largest values with no reciprocal in fp32: what is zero stays zero, nothing becomes NaN."""
    x = torch.ones(2, 256, device="cuda")
    x[:, ::2] = 0
    w = torch.full((256,), top, device="cuda")
    y8, s, _ = nm.add_rms_norm_fp8(x, w, 1e-5, group=group)
    q = y8.float()
    assert torch.all(q[:, ::2] == 0) and torch.isfinite(q).all() and torch.isfinite(s).all() and q.abs().max() <= 448
    if top > 1e-40:  # a normal maximum: the scale times e4m3's largest value gives it back
        assert torch.all(q[:, 1::2] > 0)
    if top > 1:
        assert torch.all(q[:, 1::2] == 448)


def test_offsets_past_32_bits(nm):
    """The last rows of a tensor with more than 2^31 elements, against the rows alone."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    rows, D = 1100000, 2048
    x = torch.randn(rows, D, device="cuda", dtype=torch.bfloat16)
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    y, stream = nm.add_rms_norm(x, w, residual=x)
    y8, s, _ = nm.add_rms_norm_fp8(x, w, residual=x, group=128)
    dx, _ = nm.add_rms_norm_backward(y, stream, w, d_stream=x)
    tail = x[-50:].contiguous()
    ty, ts = nm.add_rms_norm(tail, w, residual=tail)
    t8, tsc, _ = nm.add_rms_norm_fp8(tail, w, residual=tail, group=128)
    tdx, _ = nm.add_rms_norm_backward(ty, ts, w, d_stream=tail)
    assert torch.equal(y[-50:], ty) and torch.equal(stream[-50:], ts) and torch.equal(s[-50:], tsc)
    assert torch.equal(y8[-50:].view(torch.uint8), t8.view(torch.uint8)) and torch.equal(dx[-50:], tdx)


def test_in_place_stream_and_fixed_order(nm):
    import ctypes
    from state_space_model_mamba_gb300 import ssd
    x, r, dy, _, w = make(1000, 2560, torch.bfloat16, 2)
    y, stream = nm.add_rms_norm(x, w, 1e-5, residual=r)
    y2, r2 = torch.empty_like(y), r.clone()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert nm._lib().norm_add_rms(1, p(x), p(r2), p(w), 1e-5, p(y2), p(r2), 1000, 2560, ssd._stream_ptr(x.device)) == 0
    assert torch.equal(y, y2) and torch.equal(stream, r2)
    first = nm.add_rms_norm_backward(dy, stream, w)
    for a, b in zip(first, nm.add_rms_norm_backward(dy, stream, w)):
        assert torch.equal(a, b)


def test_refusals(nm):
    x, r, dy, _, w = make(4, 64, torch.bfloat16, 3)
    for bad in (dict(residual=r.float()), dict(residual=r[:2]), dict(weight=w.bfloat16()), dict(weight=w[:-1])):
        with pytest.raises(ValueError):
            nm.add_rms_norm(**dict(dict(x=x, weight=w), **bad))
    with pytest.raises(TypeError):
        nm.add_rms_norm(x.half(), w)
    with pytest.raises(ValueError):
        nm.add_rms_norm(x.t(), w)
    from state_space_model_mamba_gb300 import ssd
    with pytest.raises(ssd.SsdError):
        nm.add_rms_norm_fp8(x, w, group=48)


@pytest.mark.parametrize("group,D", [(0, 256), (128, 256), (0, 255), (0, 250), (32, 1024)])
@pytest.mark.parametrize("top", [1e-41, 1e-38, 3e-37, 1.2e-36, 6e-36, 1e-33, 0.99e-30, 1.01e-30, 1e-20])
def test_fp8_of_tiny_maxima_multiplies_back(nm, group, D, top):
    """y8 is nearest to y / scale also where the maximum's reciprocal leaves fp32 or the scale is rounded as a
    subnormal.  Half a step of e4m3 (2^-4 of the value, half of 2^-9 below 2^-6), and the two roundings on the way
    (2^-22 of the value) where that decides a tie."""
    x, _, _, _, w = make(5, D, torch.float32, D + group)
    x[3] = 0
    w = w * top
    y, _ = nm.add_rms_norm(x, w, 1e-5)
    y8, s, _ = nm.add_rms_norm_fp8(x, w, 1e-5, group=group)
    y, q, s = (t.double().cpu().numpy() for t in (y.view(5, s.shape[1], -1), y8.float().view(5, s.shape[1], -1), s))
    m = np.abs(y).max(-1)
    assert np.all(np.abs(s - m / 448) <= 2.0 ** -23 * m / 448 + 2.0 ** -150) and np.all(s[:3] > 0)
    assert np.all(q[3] == 0) and np.all(s[3] == 0)
    r = np.clip(y[:3] / s[:3, :, None], -448, 448)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -6))) - 3)
    assert np.all(np.abs(q[:3] - r) <= 0.5 * step + 2.0 ** -22 * np.abs(r))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [1e-5, 0.1])
def test_backward_of_one_column(nm, dtype, eps):
    """dx = dy w rstd (1 - (h rstd)^2), the difference of two nearly equal terms: each within 2^-20 of dy w rstd (rstd
    within two units of the last place, its square twice as far), then the result's own rounding."""
    x, _, dy, _, w = make(300, 1, dtype, 4)
    dx, dw = nm.add_rms_norm_backward(dy, x, w, eps)
    h, d, ww = (t.double().cpu().numpy() for t in (x, dy, w))
    r = 1 / np.sqrt(h * h + eps)
    ref = d * ww * eps * r ** 3
    err = np.abs(dx.double().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -20 * np.abs(d * ww * r) + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(ref))
    assert np.linalg.norm(ref) > 20 * 2.0 ** -20 * np.linalg.norm(d * ww * r)  # zeros would not do
    assert rel(dw, od.add_rms_norm_backward(d, h, ww, eps)[1]) <= 1e-5
