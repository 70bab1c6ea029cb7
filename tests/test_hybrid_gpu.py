"""The operators together, as a hybrid layer has them: the scan, the exit norm with its gate, window attention over the
normed rows, an exit norm without one -- forward, backward, and token by token from the prompt's states and rings --
against the chain of the fp64 oracles; and calls at the same time.

Bars (normwise, whole outputs): the scan's in fp32 storage is 1e-4, the others' 1e-5; what enters the softmax and the
norms moves their outputs by its relative size times a score or a normed value of a few units: 5e-4 over the chain of
four, and the same again for the chain of the gradients: 1e-3."""
import numpy as np
import pytest

import oracle
from oracle import window as ow

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

b, L, H, P, N, G, W, SINKS = 2, 150, 6, 64, 32, 2, 40, 3
D = H * P


@pytest.fixture(scope="module")
def ops():
    from state_space_model_mamba_gb300 import norm, ssd, window
    return norm, ssd, window


def inputs(seed, valid_len):
    from state_space_model_mamba_gb300.inputs import generate_small
    i = generate_small(b, L, H, P, N, G, seed=seed, init_std=0.3, d_final_std=1.0, valid_len=valid_len)
    r = np.random.default_rng(seed)
    for name, shape in (("z", (b, L, D)), ("w2", (D,)), ("dout", (b, L, D)), ("b1", (D,)), ("w1", (D,))):
        i[name] = (r.standard_normal(shape) * (0.2 if len(shape) == 1 else 1) + (1 if name[0] == "w" else 0)).astype(np.float32)
    return i


def reference(i, grads=True):
    """y of the layer, and the gradients of its inputs, in 64 bits."""
    vl = i["valid_len"]
    scan = [i[n] for n in ("x", "dt", "A", "B", "C", "D", "init")]
    s, _ = oracle.forward(*scan, vl)
    form1 = (i["w1"], i["b1"], i["z"].reshape(-1, D), H, 1e-5, True, "silu", False)
    h = ow.group_norm(s.reshape(-1, D), *form1).reshape(b, L, H, P)
    k, v = h[:, :, :G], h[:, :, G:2 * G]
    scale = P ** -0.5
    o, _ = ow.window_forward(h, k, v, W, SINKS, scale, vl)
    form2 = (i["w2"], None, None, 1, 1e-5, False, None, False)
    y, g2 = ow.group_norm(o.reshape(-1, D), *form2, dy=i["dout"].reshape(-1, D))
    y = y.reshape(b, L, D)
    if not grads:
        return y
    gw = ow.window_backward(h, k, v, g2["dx"].reshape(b, L, H, P), W, SINKS, scale, vl)
    dh = gw["dq"].copy()
    dh[:, :, :G] += gw["dk"]
    dh[:, :, G:2 * G] += gw["dv"]
    _, g1 = ow.group_norm(s.reshape(-1, D), *form1, dy=dh.reshape(-1, D))
    gs = oracle.backward(*scan, vl, g1["dx"].reshape(b, L, H, P))
    return y, dict(gs, dz=g1["dgate"].reshape(b, L, D), dw1=g1["dweight"], db1=g1["dbias"], dw2=g2["dweight"])


def cuda(i):
    return {n: torch.from_numpy(np.ascontiguousarray(a)).cuda() for n, a in i.items() if isinstance(a, np.ndarray)}


def layer(ops, d, backward=True):
    norm, ssd, window = ops
    vl = d["valid_len"]
    scan = [d[n] for n in ("x", "dt", "A", "B", "C", "D")]
    s, state = ssd.ssd_forward(*scan, 64, init_state=d["init"], valid_len=vl)
    form1 = dict(bias=d["b1"], gate=d["z"], groups=H)
    h = norm.group_norm_gated(s.view(b, L, D), d["w1"], **form1).view(b, L, H, P)
    k, v = h[:, :, :G].contiguous(), h[:, :, G:2 * G].contiguous()
    o, lse = window.window_forward(h, k, v, W, SINKS, valid_len=vl)
    form2 = dict(center=False, activation=None)
    y = norm.group_norm_gated(o.view(b, L, D), d["w2"], **form2)
    if not backward:
        return y, state, (k, v)
    g2 = norm.group_norm_gated_backward(d["dout"], o.view(b, L, D), d["w2"], **form2)
    gw = window.window_backward(h, k, v, o, lse, g2["dx"].view(b, L, H, P), W, SINKS, valid_len=vl)
    dh = gw["dq"]
    dh[:, :, :G] += gw["dk"]
    dh[:, :, G:2 * G] += gw["dv"]
    g1 = norm.group_norm_gated_backward(dh.view(b, L, D), s.view(b, L, D), d["w1"], **form1)
    gs = ssd.ssd_backward(*scan, 64, g1["dx"].view(b, L, H, P), init_state=d["init"], valid_len=vl)
    return y, dict(gs, dz=g1["dgate"], dw1=g1["dweight"], db1=g1["dbias"], dw2=g2["dweight"])


def rel(got, ref):
    got = got.double().cpu().numpy()
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("valid_len", [[L, L], [97, 1]])
def test_a_layer_and_its_gradients(ops, valid_len):
    i = inputs(31, valid_len)
    ry, rg = reference(i)
    y, g = layer(ops, cuda(i))
    torch.cuda.synchronize()
    assert rel(y, ry) <= 5e-4
    for name in ("dx", "ddt", "dA", "dB", "dC", "dD", "d_init", "dz", "dw1", "db1", "dw2"):
        assert rel(g[name], rg[name]) <= 1e-3, name
    for r, V in enumerate(valid_len):  # nothing comes out of absent tokens
        assert not y[r, V:].any() and not g["dx"][r, V:].any() and not g["dz"][r, V:].any()


def test_a_layer_in_a_graph_has_the_same_bits(ops):
    d = cuda(inputs(32, [L, 60]))
    y, g = layer(ops, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = layer(ops, d)
    for _ in range(2):
        y2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_tokens_after_prompts_are_the_sequence(ops):
    norm, ssd, window = ops
    i = inputs(33, None)
    i["valid_len"] = None
    ref = reference(i, grads=False)
    lengths = torch.tensor([120, 33], dtype=torch.int32, device="cuda")
    d = dict(cuda(i), valid_len=lengths)
    _, state, (k, v) = layer(ops, d, backward=False)
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    states = torch.full((4, H, P, N), float("nan"), device="cuda")
    states[slots.long()] = state
    rings = [torch.full((4, SINKS + W, G, P), float("nan"), device="cuda") for _ in range(2)]
    window.window_fill(k, v, *rings, W, SINKS, valid_len=lengths, cache_index=slots)
    rows = torch.arange(b, device="cuda")
    for t in range(25):
        at = (lengths + t).long()
        s = ssd.ssd_step(d["x"][rows, at], d["dt"][rows, :, at].contiguous(), d["A"], d["B"][rows, at], d["C"][rows, at], d["D"],
                         states, state_index=slots)
        h = norm.group_norm_gated(s.view(b, D), d["w1"], bias=d["b1"], gate=d["z"][rows, at], groups=H).view(b, H, P)
        o = window.window_step(h, h[:, :G].contiguous(), h[:, G:2 * G].contiguous(), *rings, lengths + t, W, SINKS, cache_index=slots)
        y = norm.group_norm_gated(o.view(b, D), d["w2"], center=False, activation=None)
        assert rel(y, ref[np.arange(b), at.cpu().numpy()]) <= 5e-4, t
    for free in (1, 3):
        assert torch.isnan(states[free]).all() and torch.isnan(rings[0][free]).all()


def test_calls_at_the_same_time(ops):
    """Two streams with layers of different lengths, started while the other runs, give the bits of either alone."""
    ds = [cuda(inputs(34, [L, 70])), cuda(inputs(35, [20, L]))]
    alone = [layer(ops, d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(5):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append(layer(ops, d))
        torch.cuda.synchronize()
        for (y, g), (y2, g2) in zip(alone, got):
            assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("B,T,Hq,Gk,P_,Wn,sinks,valid", [
    (1, 6000, 24, 8, 128, 1024, 4, None), (3, 3500, 12, 12, 128, 200, 130, [3500, 0, 2999]), (2, 5000, 16, 4, 64, 700, 0, [5000, 4097]),
    (2, 4500, 16, 1, 40, 64, 1, [1, 4500])])
def test_more_tiles_than_blocks(ops, B, T, Hq, Gk, P_, Wn, sinks, valid):
    """Every resident block takes several tiles, of different lengths: the tensor cores' kernels against those on CUDA
    cores (held to the oracle in test_window_gpu.py): two bars of 2^-8, the second's own error being below the first's."""
    window = ops[2]
    g = torch.Generator(device="cuda").manual_seed(B + T)
    q, do = (torch.randn(B, T, Hq, P_, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(B, T, Gk, P_, generator=g, device="cuda").bfloat16() for _ in range(2))
    vl = None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")
    o, lse = window.window_forward(q, k, v, Wn, sinks, valid_len=vl, check_status=True)
    got = window.window_backward(q, k, v, o, lse, do, Wn, sinks, valid_len=vl, check_status=True)
    ro, rl = window.window_forward(q, k, v, Wn, sinks, valid_len=vl, simt=True)
    ref = window.window_backward(q, k, v, ro, rl, do, Wn, sinks, valid_len=vl, simt=True)
    # lse's scores are sums of P products in fp32 in another order
    assert (lse - rl).norm() <= 1e-5 * rl.norm()
    for name, a, r in [("o", o, ro)] + [(n, got[n], ref[n]) for n in ("dq", "dk", "dv")]:
        a, r = a.float(), r.float()
        assert (a - r).norm() <= 2.0 ** -7 * r.norm(), name
        rows, floor = r.flatten(0, 1).norm(dim=(1, 2)), 0.1 * r.norm() / (B * T) ** 0.5
        off = (a - r).flatten(0, 1).norm(dim=(1, 2))
        assert (off <= 4 * 2.0 ** -7 * rows.clamp_min(floor)).all(), name
    again = window.window_backward(q, k, v, o, lse, do, Wn, sinks, valid_len=vl)
    assert all(torch.equal(again[n], got[n]) for n in got)
