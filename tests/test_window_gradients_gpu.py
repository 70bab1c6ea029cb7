"""Gradients of window attention (include/window.h) on the GPU, against the 64-bit definition with the o that the backward was given
(tests/window_util.py derives the bars): every shape, scales of every size and sign, tensors past 2^31 elements; and the
one-token step at other scales."""
import numpy as np
import pytest
import window_util as wu

from oracle import window as ow

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FORMS = [(False, False), (True, False), (True, True)]  # bf16, simt


@pytest.fixture(scope="module")
def wd():
    from state_space_model_mamba_gb300 import window
    return window


def dev(a, bf16):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.bfloat16 if bf16 else torch.float32)


def ints(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def host(t):
    return t.double().cpu().numpy()


def train(wd, d, W, sinks, **kw):
    o, lse = wd.window_forward(d["q"], d["k"], d["v"], W, sinks, **kw)
    return dict(wd.window_backward(d["q"], d["k"], d["v"], o, lse, d["do"], W, sinks, **kw), o=o, lse=lse)


def compare(wd, x, W, sinks, bf16, simt, scale=None, valid=None, extra=0.0):
    out = train(wd, {n: dev(a, bf16) for n, a in x.items()}, W, sinks, scale=scale, valid_len=ints(valid), simt=simt)
    torch.cuda.synchronize()
    c = x["q"].shape[-1] ** -0.5 if scale is None else scale
    ref = ow.window_backward(x["q"], x["k"], x["v"], x["do"], W, sinks, c, valid, o=host(out["o"]))
    for name, r in ref.items():
        wu.check(host(out[name]), r, (wu.BF16_BAR if bf16 else wu.F32_BAR) + extra, name)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("b,L,H,G,P,W,sinks", wu.SHAPES)
def test_bf16(wd, b, L, H, G, P, W, sinks, simt):
    compare(wd, wu.draw(b, L, H, G, P, L + W), W, sinks, True, simt)


@pytest.mark.parametrize("b,L,H,G,P,W,sinks", wu.F32_SHAPES)
def test_f32(wd, b, L, H, G, P, W, sinks):
    compare(wd, wu.draw(b, L, H, G, P, L + W, False), W, sinks, False, False)


@pytest.mark.parametrize("bf16,simt", FORMS)
@pytest.mark.parametrize("scale", [30.0, -30.0, 1.0, -0.125, 1e-3, -1e-30, 0.0])
def test_scales_of_every_size(wd, bf16, simt, scale):
    """Rows of a single key, of all keys alike, and negative scales.  A score of size s is off by some 2^-23 s (a sum of 64 exact products
    in fp32, lse's rounding), which is what p and dx are off by, relative: 8 times that on top of the bar."""
    x, valid = wu.draw(2, 260, 4, 2, 64, 12, bf16), [260, 201]
    lse = ow.window_forward(x["q"], x["k"], x["v"], 70, 3, scale, valid)[1]
    compare(wd, x, 70, 3, bf16, simt, scale, valid, 8 * max(1.0, np.abs(lse).max()) * 2.0 ** -23)


@pytest.mark.parametrize("bf16,P", [(False, 64), (True, 64), (True, 20)])
@pytest.mark.parametrize("scale", [30.0, -30.0, 1e-3, -0.5, 0.0])
def test_step_at_other_scales(wd, bf16, P, scale):
    """Scores are off as above; rings full, young and with a token alone."""
    b, H, G, W, sinks = 4, 10, 2, 90, 3
    x, r = wu.draw(b, 1, H, G, P, 17, bf16), np.random.default_rng(18)
    kc, vc = (wu.store(r.standard_normal((b + 1, sinks + W, G, P)), bf16) for _ in range(2))
    pos, index = [1000, 40, 0, sinks + W - 1], [4, 0, 2, 1]
    o = wd.window_step(*(dev(x[n][:, 0], bf16) for n in "qkv"), dev(kc, bf16), dev(vc, bf16), ints(pos), W, sinks, scale=scale,
                       cache_index=ints(index))
    ro, rk, _ = ow.window_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], kc, vc, pos, W, sinks, scale, index)
    s = abs(scale) * max(np.abs(rk[i, :, h // 5] @ x["q"][n, 0, h]).max() for n, i in enumerate(index) for h in range(H))
    wu.check(host(o), ro, (wu.BF16_BAR if bf16 else wu.F32_BAR) + 8 * max(1.0, s) * 2.0 ** -23, "o", 2)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("G", [6, 192])
def test_offsets_past_32_bits(wd, bf16, G):
    """q, o, do and dq (with 192 key heads also k, v, dk and dv) of 2.4e9 elements: the last row's outputs are those of a call on it
    alone, bit for bit (sums have one order, whatever else is in the batch)."""
    b, L, H, P, W, sinks = 3, 32768, 192, 128, 64, 2
    if torch.cuda.mem_get_info()[0] < (2 if bf16 else 4) * b * L * P * (5 * H + 7 * G) + (20 << 30):
        pytest.skip("needs more memory")
    T = torch.bfloat16 if bf16 else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(G)
    d = {n: torch.empty(b, L, h, P, device="cuda", dtype=T) for n, h in (("q", H), ("k", G), ("v", G), ("do", H))}
    for t in d.values():
        for row in t:
            row.copy_(torch.randn(row.shape, generator=gen, device="cuda", dtype=T))
    valid = [L, L // 3, L - 77]
    whole = train(wd, d, W, sinks, valid_len=ints(valid))
    last = {n: t[-1:].clone() for n, t in whole.items()}
    del whole
    alone = train(wd, {n: t[-1:].clone() for n, t in d.items()}, W, sinks, valid_len=ints(valid[-1:]))
    for n in alone:
        assert torch.equal(last[n], alone[n]), n
    assert alone["dq"][0, 1:valid[-1]].abs().amax((1, 2)).min() > 0  # every token that sees another has a gradient


def scaled_alike(wd, bf16, simt, power):
    """The outputs at q, k and a scale, and at q and k times 2^power and the scale times 2^-2power: the same scores, exactly."""
    x = wu.draw(1, 300, 4, 2, 64, 31, bf16)
    big = dict(x, q=x["q"] * np.float32(2.0 ** power), k=x["k"] * np.float32(2.0 ** power))
    for sign in (1, -1):
        yield [train(wd, {n: dev(t, bf16) for n, t in y.items()}, 70, 3, scale=sign * s, simt=simt)
               for y, s in ((x, 0.125), (big, 2.0 ** (-3 - 2 * power)))]


@pytest.mark.parametrize("bf16,simt", FORMS)
@pytest.mark.parametrize("power", [53, 60])
def test_tiny_scales_of_large_scores(wd, bf16, simt, power):
    """o, lse and dv are the same bit for bit."""
    for a, b in scaled_alike(wd, bf16, simt, power):
        for n in ("o", "lse", "dv"):
            assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("bf16,simt", FORMS)
@pytest.mark.parametrize("power", [53, 60])
def test_gradients_at_tiny_scales(wd, bf16, simt, power):
    """dq and dk are the same times 2^-power, bit for bit while that is a normal number."""
    for a, b in scaled_alike(wd, bf16, simt, power):
        for n in ("dq", "dk"):
            ok = a[n].float().abs() >= 2.0 ** (power - 120)
            assert torch.equal((a[n].float() * 2.0 ** -power)[ok], b[n].float()[ok]), n
