"""Pins of oracle/window.py (no GPU): gradients against central differences, the ring against the sequence,
the window against plain causal attention, and the step of the scan against the scan's own oracle."""
import numpy as np
import pytest

import oracle
from oracle import window as ow


def draw(b, L, H, G, P, seed):
    r = np.random.default_rng(seed)
    return (r.standard_normal((b, L, H, P)), r.standard_normal((b, L, G, P)), r.standard_normal((b, L, G, P)),
            r.standard_normal((b, L, H, P)))


@pytest.mark.parametrize("window,sinks,valid", [(3, 0, None), (4, 2, [9, 6]), (1, 1, [0, 10]), (20, 3, [10, 1])])
def test_gradients_against_differences(window, sinks, valid):
    q, k, v, do = draw(2, 10, 4, 2, 5, 1)
    g = ow.window_backward(q, k, v, do, window, sinks, 0.4, valid)
    r = np.random.default_rng(2)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        d, h = r.standard_normal(x.shape), 1e-5
        vals = []
        for sign in (1, -1):
            y = x + sign * h * d
            args = {"dq": (y, k, v), "dk": (q, y, v), "dv": (q, k, y)}[name]
            vals.append(float((ow.window_forward(*args, window, sinks, 0.4, valid)[0] * do).sum()))
        assert abs((vals[0] - vals[1]) / (2 * h) - float((g[name] * d).sum())) < 1e-7 * max(1.0, np.linalg.norm(g[name]))
        if valid is not None:
            for i, V in enumerate(valid):
                assert not g[name][i, V:].any()


def test_wide_window_is_causal_attention():
    q, k, v, _ = draw(1, 12, 2, 2, 4, 3)
    o, lse = ow.window_forward(q, k, v, 12, 0, 0.5)
    for h in range(2):
        x = 0.5 * q[0, :, h] @ k[0, :, h].T
        x = np.where(np.tril(np.ones((12, 12))) > 0, x, -np.inf)
        e = np.exp(x)
        assert np.allclose(o[0, :, h], (e / e.sum(1, keepdims=True)) @ v[0, :, h], atol=1e-13)
        assert np.allclose(lse[0, h], np.log(e.sum(1)), atol=1e-13)
    a = ow.window_forward(q, k, v, 5, 12, 0.5)[0]  # every token a sink: the same
    assert np.allclose(a, o, atol=1e-13)


@pytest.mark.parametrize("window,sinks", [(4, 0), (3, 2), (1, 3), (30, 2)])
def test_steps_through_the_ring_are_the_sequence(window, sinks):
    q, k, v, _ = draw(2, 17, 4, 2, 5, 4)
    o, _ = ow.window_forward(q, k, v, window, sinks, 0.4)
    lengths, index = [6, 0], [2, 0]
    shape = (3, sinks + window, 2, 5)
    kc, vc = np.full(shape, np.nan), np.full(shape, np.nan)
    kc = ow.window_fill(k[:, :8], kc, window, sinks, lengths, index)
    vc = ow.window_fill(v[:, :8], vc, window, sinks, lengths, index)
    for t in range(9):
        pos = [x + t for x in lengths]
        rows = [0, 1]
        got, kc, vc = ow.window_step(q[rows, pos], k[rows, pos], v[rows, pos], kc, vc, pos, window, sinks, 0.4, index)
        assert np.allclose(got, o[rows, pos], atol=1e-13)
    assert np.isnan(kc[1]).all()


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate,first", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
def test_group_norm_gradients_against_differences(activation, gate, first, center):
    r = np.random.default_rng(5)
    x, z, w, bias, dy = (r.standard_normal(s) for s in ((3, 12), (3, 12), 12, 12, (3, 12)))
    z = z if gate else None
    form = (3, 1e-2, center, activation, first)
    _, g = ow.group_norm(x, w, bias, z, *form, dy=dy)
    leaves = dict(dx=x, dweight=w, dbias=bias, **({"dgate": z} if gate else {}))
    for name, a in leaves.items():
        d, h, vals = r.standard_normal(a.shape), 1e-5, []
        for sign in (1, -1):
            y = dict(leaves, **{name: a + sign * h * d})
            vals.append(float((ow.group_norm(y["dx"], y["dweight"], y["dbias"], y.get("dgate"), *form) * dy).sum()))
        assert abs((vals[0] - vals[1]) / (2 * h) - float((g[name] * d).sum())) < 1e-7 * max(1.0, np.linalg.norm(g[name]))
    assert (g["dgate"] is None) == (not gate)


def test_scan_steps_are_the_scan():
    r = np.random.default_rng(6)
    b, L, H, P, N, G = 2, 5, 4, 3, 4, 2
    f = np.float32
    x, B, C = (r.standard_normal(s).astype(f) for s in ((b, L, H, P), (b, L, G, N), (b, L, G, N)))
    dt, A, D = r.random((b, H, L)).astype(f), -r.random(H).astype(f), r.standard_normal(H).astype(f)
    init = r.standard_normal((b, H, P, N)).astype(f)
    y, fin = oracle.forward(x, dt, A, B, C, D, init, None)
    pool, index = np.zeros((5, H, P, N)), [3, 1]
    pool[index] = init
    for t in range(L):
        got, pool = ow.ssd_step(x[:, t], dt[:, :, t], A, B[:, t], C[:, t], D, pool, index)
        assert np.allclose(got, y[:, t], atol=1e-6)
    assert np.allclose(pool[index], fin, atol=1e-6) and not pool[[0, 2, 4]].any()
    got, after = ow.ssd_step(x[:, 0], dt[:, :, 0], A, B[:, 0], C[:, 0], D, pool, [5, -1])
    assert not got.any() and (after == pool).all()
