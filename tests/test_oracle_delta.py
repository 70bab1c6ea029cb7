"""The fp64 oracle of the gated delta rule and of the entry norm, pinned on the
CPU: finite differences for every gradient, and closed forms of special cases."""
import numpy as np
import pytest

from oracle import delta as od


def inputs(seed=0, b=2, L=7, H=4, P=3, N=5, G=2):
    r = np.random.default_rng(seed)
    k = r.standard_normal((b, L, G, N))
    return dict(q=r.standard_normal((b, L, G, N)), k=k / np.linalg.norm(k, axis=-1, keepdims=True),
                v=r.standard_normal((b, L, H, P)), g=-r.exponential(0.3, (b, H, L)), beta=r.uniform(0, 1, (b, H, L)),
                init=r.standard_normal((b, H, P, N)), do=r.standard_normal((b, L, H, P)),
                d_final=r.standard_normal((b, H, P, N)))


def loss(x, scale, valid):
    o, S = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["init"], valid)
    return (x["do"] * o).sum() + (x["d_final"] * S).sum()


@pytest.mark.parametrize("valid", [None, [7, 0], [1, 5]])
def test_gradients_against_central_differences(valid):
    x, scale = inputs(), 0.7
    gr = od.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["do"], x["d_final"], x["init"], valid)
    r = np.random.default_rng(1)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("init", "d_init")):
        for _ in range(3):
            u = r.standard_normal(x[name].shape)
            h = 1e-6
            hi, lo = (loss(dict(x, **{name: x[name] + s * h * u}), scale, valid) for s in (1, -1))
            # central difference of a function of order 10: truncation h^2, rounding 1e-15 * 10 / h
            assert abs((hi - lo) / (2 * h) - (gr[grad] * u).sum()) < 1e-6 * (1 + np.abs(gr[grad] * u).sum()), name


def test_full_write_reads_back_the_value():
    # beta = 1, unit key: the state answers the key with exactly the last value written for it
    x = inputs(3)
    x["beta"][:] = 1.0
    o, _ = od.delta_forward(x["k"], x["k"], x["v"], x["g"], x["beta"], 1.0, x["init"])
    np.testing.assert_allclose(o, x["v"], rtol=0, atol=1e-12)


def test_beta_zero_only_decays():
    x = inputs(4)
    x["beta"][:] = 0.0
    _, S = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 1.0, x["init"])
    np.testing.assert_allclose(S, x["init"] * np.exp(x["g"].sum(-1))[..., None, None], rtol=1e-12)


def test_steps_equal_the_sequence():
    x = inputs(5)
    o, S = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["init"])
    state = np.concatenate([x["init"], np.zeros((1,) + x["init"].shape[1:])])
    for t in range(7):
        step = od.delta_step(x["q"][:, t], x["k"][:, t], x["v"][:, t], x["g"][:, :, t], x["beta"][:, :, t], 0.5, state,
                             np.array([1, 0]) if t < 0 else None)
        np.testing.assert_allclose(step, o[:, t], atol=1e-12)
    np.testing.assert_allclose(state[:2], S, atol=1e-12)


def test_norm_gradient_against_central_differences():
    r = np.random.default_rng(6)
    h, dy, w, ds = r.standard_normal((3, 10)), r.standard_normal((3, 10)), r.standard_normal(10), r.standard_normal((3, 10))
    dx, dw = od.add_rms_norm_backward(dy, h, w, 1e-5, ds)
    e = 1e-6
    u, uw = r.standard_normal(h.shape), r.standard_normal(10)
    f = lambda hh, ww: (od.add_rms_norm(hh, ww, 1e-5) * dy).sum() + (ds * hh).sum()  # noqa: E731
    assert abs((f(h + e * u, w) - f(h - e * u, w)) / (2 * e) - (dx * u).sum()) < 1e-7
    assert abs((f(h, w + e * uw) - f(h, w - e * uw)) / (2 * e) - (dw * uw).sum()) < 1e-7


def test_steps_through_slots_in_any_order():
    """Requests keep their slots of a larger pool, one is absent at every step; the other slots are left alone."""
    x = inputs(7)
    o, S = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["init"])
    r = np.random.default_rng(8)
    state = r.standard_normal((5,) + x["init"].shape[1:])
    state[3], state[0] = x["init"][0], x["init"][1]
    before = state.copy()
    for t in range(7):
        order, index = (np.array([1, 0, 0]), np.array([0, 3, -1])) if t % 2 else (np.array([0, 1, 1]), np.array([3, 0, 5]))
        step = od.delta_step(*(x[n][order, t] for n in ("q", "k", "v")), *(x[n][order, :, t] for n in ("g", "beta")), 0.5, state, index)
        np.testing.assert_allclose(step[:2], o[order[:2], t], atol=1e-12)
        assert np.all(step[2] == 0)
    np.testing.assert_allclose(state[[3, 0]], S, atol=1e-12)
    np.testing.assert_array_equal(state[[1, 2, 4]], before[[1, 2, 4]])
