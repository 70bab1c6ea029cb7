"""The comparison that the gradients of window attention are held to (tests/window_util.py), on the CPU: at every shape it takes the
definition with the tensor-core kernels' roundings, and refuses gradients that are 1 % off in their size or in do . o."""
import numpy as np
import pytest
import window_util as wu

from oracle import window as ow


def rounded_backward(x, W, sinks, scale, o):
    """The definition with p and dx rounded to bf16 where they enter a product, and outputs rounded once."""
    q, k, v, do = (x[n].astype(np.float64) for n in ("q", "k", "v", "do"))
    (b, L, H, P), G = q.shape, k.shape[2]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for i in range(b):
        for t in range(L):
            s = ow.seen(t, W, sinks)
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                y = scale * q[i, t, hs] @ k[i, s, g].T
                p = np.exp(y - y.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                D = (do[i, t, hs] * o[i, t, hs]).sum(-1, keepdims=True)
                dx = wu.store(p * (do[i, t, hs] @ v[i, s, g].T - D), True).astype(np.float64)
                dq[i, t, hs] = scale * dx @ k[i, s, g]
                dk[i, s, g] += scale * dx.T @ q[i, t, hs]
                dv[i, s, g] += wu.store(p, True).astype(np.float64).T @ do[i, t, hs]
    return {n: wu.store(a, True) for n, a in (("dq", dq), ("dk", dk), ("dv", dv))}


@pytest.mark.parametrize("b,L,H,G,P,W,sinks", wu.SHAPES)
def test_the_comparison_takes_roundings_and_refuses_one_percent(b, L, H, G, P, W, sinks):
    x, scale = wu.draw(b, L, H, G, P, L + W), P ** -0.5
    o = wu.store(ow.window_forward(x["q"], x["k"], x["v"], W, sinks, scale)[0], True)
    args = (x["q"], x["k"], x["v"], x["do"], W, sinks, scale)
    ref = ow.window_backward(*args, o=o)
    good, off = rounded_backward(x, W, sinks, scale, o), ow.window_backward(*args, o=1.01 * o)
    for name in ("dq", "dk", "dv"):
        wu.check(good[name], ref[name], wu.BF16_BAR, name)
        with pytest.raises(AssertionError, match=name):
            wu.check(1.01 * ref[name], ref[name], wu.BF16_BAR, name)
    for name in ("dq", "dk"):
        with pytest.raises(AssertionError, match=name):
            wu.check(off[name], ref[name], wu.BF16_BAR, name)


def test_a_given_o_is_used():
    x = wu.draw(1, 9, 2, 1, 8, 1)
    o = ow.window_forward(x["q"], x["k"], x["v"], 4, 1, 0.3)[0]
    a, b = (ow.window_backward(x["q"], x["k"], x["v"], x["do"], 4, 1, 0.3, **kw) for kw in ({}, dict(o=o)))
    for name in a:
        np.testing.assert_allclose(a[name], b[name], rtol=0, atol=1e-13)


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_scales_past_fp32_in_base_2_are_refused(scale):
    """A scale whose product with log2(e) overflows would make every score infinite."""
    import ctypes
    from state_space_model_mamba_gb300 import build, ssd, window
    build.build()
    lib, buf = window._lib(), ctypes.c_void_p(1 << 20)  # never dereferenced: the calls fail before a launch
    d = [ctypes.byref(window.WindowDims(2, n, 4, 64, 2, 16, 4, 0, 0)) for n in (100, 1)]
    for code in (0, 1):
        assert lib.window_forward(d[0], code, buf, buf, buf, scale, None, buf, None, buf, 1 << 40, None) == ssd.SSD_ERR_INVALID_ARG
        assert b"finite" in lib.ssd_last_error()
        assert lib.window_backward(d[0], code, *([buf] * 6 + [scale, None] + [buf] * 4 + [1 << 40, None])) == ssd.SSD_ERR_INVALID_ARG
        assert lib.window_step(d[1], code, buf, buf, buf, buf, scale, buf, buf, 2, None, buf, None) == ssd.SSD_ERR_INVALID_ARG
