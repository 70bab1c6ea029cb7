"""GPU parity of the gated delta rule (include/delta.h), through the C ABI,
against the token-by-token fp64 oracle (oracle/delta.py).

Bars, as normwise relative errors of whole outputs:
  * fp32 storage: a handful of fp32 roundings (2^-24) a token over the at most
    ~100 tokens that a contracting state remembers, and sums over N <= 256: 1e-5;
  * bf16 storage, bf16 outputs: one rounding at the end (2^-8 at most, 1.7e-3
    root-mean-square) and operands rounded once on the way (as much again, in
    quadrature): 2^-8;
  * bf16 storage, fp32 outputs (final_state, dg, dbeta, d_init): operands held
    as two bf16 (2^-17 off at most) through three chained products: 3 * 2^-17.
Slices along the leading axes are held to four times the bar, their norms
floored at a tenth of the tensor's RMS slice norm."""
import numpy as np
import pytest

from oracle import delta as od

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32_BAR, BF16_BAR, SPLIT_BAR = 1e-5, 2.0 ** -8, 3 * 2.0 ** -17


@pytest.fixture(scope="module")
def dl():
    from state_space_model_mamba_gb300 import delta
    return delta


def draw(b, L, H, P, N, G, seed, dt_mu=-3.0, bf16=True, relu_keys=False):
    r = np.random.default_rng(seed)

    def store(x):
        t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
        return t.bfloat16().float().numpy() if bf16 else t.numpy()

    def unit(x):
        x = np.maximum(x, 0.05) if relu_keys else x / (1 + np.exp(-x))
        return store(x / np.linalg.norm(x, axis=-1, keepdims=True))

    f = np.float32
    return dict(q=unit(r.standard_normal((b, L, G, N))), k=unit(r.standard_normal((b, L, G, N))),
                v=store(r.standard_normal((b, L, H, P))),
                g=(-np.exp(r.uniform(0, np.log(16), H))[None, :, None]
                   * np.logaddexp(0, r.standard_normal((b, H, L)) + dt_mu)).astype(f),
                beta=(1 / (1 + np.exp(-r.standard_normal((b, H, L))))).astype(f),
                init=(0.3 * r.standard_normal((b, H, P, N))).astype(f), do=store(r.standard_normal((b, L, H, P))),
                d_final=r.standard_normal((b, H, P, N)).astype(f))


def dev(x, bf16):
    T = torch.bfloat16 if bf16 else torch.float32
    return {k: torch.from_numpy(a).cuda().to(T if k in ("q", "k", "v", "do") else torch.float32) for k, a in x.items()}


def check(got, ref, bar, what, axes):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    d = got - ref
    n = np.linalg.norm(ref)
    whole = np.linalg.norm(d) / n if n else np.linalg.norm(d)
    assert whole <= bar, f"{what}: {whole:.3e} > {bar:.3e}"
    m = int(np.prod(ref.shape[:axes]))
    rn = np.linalg.norm(ref.reshape(m, -1), axis=1)
    floor = max(0.1 * np.sqrt(np.mean(rn ** 2)), 1e-30)
    worst = np.max(np.linalg.norm(d.reshape(m, -1), axis=1) / np.maximum(rn, floor))
    assert worst <= 4 * bar, f"{what}, worst slice: {worst:.3e} > {4 * bar:.3e}"


def run(dl, x, bf16, scale, init=True, valid=None, backward=True, simt=False, d_final=True):
    d = dev(x, bf16)
    vl = None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")
    a = (d["q"], d["k"], d["v"], d["g"], d["beta"])
    out = dict(zip(("o", "final"), dl.delta_forward(*a, scale=scale, init_state=d["init"] if init else None,
                                                    valid_len=vl, simt=simt)))
    if backward:
        out.update(dl.delta_backward(*a, d["do"], scale=scale, d_final_state=d["d_final"] if d_final else None,
                                     init_state=d["init"] if init else None, valid_len=vl, simt=simt))
    torch.cuda.synchronize()
    return out


def compare(out, x, bf16, scale, init=True, valid=None, d_final=True, split=True):
    ini = x["init"] if init else None
    o, S = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, ini, valid)
    ref = dict(o=o, final=S)
    if "dq" in out:
        ref.update(od.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["do"],
                                     x["d_final"] if d_final else None, ini, valid))
    for name, r in ref.items():
        stored = name in ("o", "dq", "dk", "dv")
        bar = F32_BAR if not bf16 else (BF16_BAR if stored else SPLIT_BAR)
        check(out[name], r, bar, name, 2 if not stored else 3)


# one token, chunk edges, ragged tails; padded and full key and value widths; shared and own keys
SHAPES = [(1, 1, 1, 64, 128, 1), (2, 63, 2, 64, 64, 1), (1, 64, 4, 128, 128, 2), (2, 65, 2, 64, 128, 2),
          (1, 130, 6, 96, 80, 2), (3, 200, 2, 8, 8, 1), (1, 257, 3, 128, 64, 3), (1, 700, 2, 64, 128, 1)]


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_bf16_forward_backward(dl, shape, simt):
    x = draw(*shape, seed=sum(shape))
    scale = shape[4] ** -0.5
    compare(run(dl, x, True, scale, simt=simt), x, True, scale)


@pytest.mark.parametrize("shape", [(1, 1, 1, 4, 4, 1), (2, 37, 4, 12, 20, 2), (1, 100, 2, 128, 256, 1), (2, 70, 3, 36, 132, 3),
                                   (1, 300, 2, 64, 128, 2), (2, 33, 2, 100, 196, 1)])
@pytest.mark.parametrize("init", [True, False])
def test_f32_forward_backward(dl, shape, init):
    x = draw(*shape, seed=7 + sum(shape), bf16=False)
    compare(run(dl, x, False, 0.5, init=init), x, False, 0.5, init=init)


@pytest.mark.parametrize("shape, valid", [((2, 37, 80, 8, 12, 4), [37, 5]), ((1, 21, 80, 40, 196, 2), None), ((4, 18, 40, 12, 100, 5), [0, 18, 1, 17])])
def test_f32_more_heads_than_blocks_of_few_rows(dl, shape, valid):
    x = draw(*shape, seed=sum(shape), bf16=False)
    compare(run(dl, x, False, 0.5, valid=valid), x, False, 0.5, valid=valid)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("valid", [[150, 0, 1], [64, 128, 149], [63, 65, 2]])
def test_valid_len_and_garbage_past_it(dl, bf16, valid):
    x = draw(3, 150, 4, 64, 128, 2, seed=3, bf16=bf16)
    y = {k: a.copy() for k, a in x.items()}
    for i, n in enumerate(valid):  # absent tokens hold what must not be read into anything
        for k in ("q", "k", "v", "do"):
            y[k][i, n:] = np.nan
        y["g"][i, :, n:], y["beta"][i, :, n:] = np.inf, np.nan
    out = run(dl, y, bf16, 0.3, valid=valid)
    compare(out, x, bf16, 0.3, valid=valid)
    for i, n in enumerate(valid):
        for k in ("o", "dq", "dk", "dv"):
            assert torch.all(out[k][i, n:] == 0), k
        for k in ("dg", "dbeta"):
            assert torch.all(out[k][i, :, n:] == 0), k


@pytest.mark.parametrize("shape, valid", [((5, 300, 40, 64, 64, 8), None), ((4, 420, 48, 40, 128, 16), [420, 0, 65, 192]),
                                          ((2, 190, 90, 128, 32, 90), [1, 190]), ((200, 70, 1, 64, 64, 1), None),
                                          ((2, 130, 160, 8, 16, 2), None)])
def test_more_chains_than_blocks_run_at_once(dl, shape, valid):
    x = draw(*shape, seed=sum(shape))
    compare(run(dl, x, True, 0.3, valid=valid), x, True, 0.3, valid=valid)


def test_halves_of_the_batch_on_two_streams(dl):
    """More chains than SMs over 16 chunks and more: the backward forks.  Ordered on the caller's stream, the
    same bits when captured and replayed."""
    valid = [1030, 0, 700]
    x = draw(3, 1030, 64, 8, 8, 2, seed=8)
    out = run(dl, x, True, 0.3, valid=valid)
    compare(out, x, True, 0.3, valid=valid)
    d = dev(x, True)
    vl = torch.tensor(valid, dtype=torch.int32, device="cuda")
    a = (d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"])
    kw = dict(scale=0.3, d_final_state=d["d_final"], init_state=d["init"], valid_len=vl)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        late = torch.empty_like(d["do"])
        torch.cuda._sleep(2_000_000)
        late.copy_(d["do"])  # the fork has to come after this, the join before the copies below
        got = dl.delta_backward(*a[:5], late, **kw)
        copies = {k: t.clone() for k, t in got.items()}
    torch.cuda.current_stream().wait_stream(other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=other):
        captured = dl.delta_backward(*a, **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in copies:
        assert torch.equal(copies[k], got[k]) and torch.equal(captured[k], got[k]), k
        if k in out:
            assert torch.equal(out[k], got[k]), k


def large(b, L, H, P, N, G, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def unit(x):
        return torch.nn.functional.normalize(x, dim=-1)

    return dict(q=unit(rand(b, L, G, N)), k=unit(rand(b, L, G, N)), v=rand(b, L, H, P),
                g=-torch.rand(b, H, L, generator=g, device="cuda"), beta=torch.rand(b, H, L, generator=g, device="cuda"))


def near(a, b, bar):
    """Rows that take another grid: the same sums, grouped differently."""
    assert a.shape == b.shape and torch.isfinite(a).all()
    assert float((a.float() - b.float()).norm()) <= bar * float(b.float().norm())


def test_offsets_past_32_bits(dl):
    """The last rows of tensors with more than 2^31 elements, and of workspaces past 4 GB, against the rows alone."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    t = large(3, 131072, 64, 128, 32, 1, 1)
    assert t["v"].numel() > 2 ** 31
    o, fin = dl.delta_forward(*t.values())
    last = {k: x[2:].contiguous() for k, x in t.items()}
    del t
    o, fin = o[2:].clone(), fin[2:].clone()
    ro, rf = dl.delta_forward(*last.values())
    near(o, ro, BF16_BAR)
    near(fin, rf, SPLIT_BAR)
    del o, ro, last
    t = large(2, 32768, 80, 64, 128, 16, 2)
    do = torch.randn_like(t["v"])
    out = dl.delta_backward(*t.values(), do)
    ref = dl.delta_backward(*(x[1:].contiguous() for x in t.values()), do[1:].contiguous())
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(out[k][1:], ref[k]), k  # halves of the batch: the same kernels
    del out, ref, do, t
    slots, H, P, N = 4200, 80, 64, 128
    pool = torch.zeros(slots, H, P, N, device="cuda")
    assert pool.numel() > 2 ** 31
    x = large(2, 1, H, P, N, 16, 3)
    pool[-1], pool[1] = 0.25, 0.25
    index = torch.tensor([slots - 1, 1], dtype=torch.int32, device="cuda")
    one = [y[:1].expand_as(y).squeeze(2 if n in ("g", "beta") else 1).contiguous() for n, y in x.items()]
    o = dl.delta_step(*one, pool, state_index=index)
    assert torch.equal(o[0], o[1]) and torch.equal(pool[-1], pool[1]) and float((pool[1] - 0.25).abs().max()) > 1e-3
    assert float(pool[2:-1].abs().max()) == 0 and float(pool[0].abs().max()) == 0


@pytest.mark.parametrize("bf16", [True, False])
def test_no_state_no_final_gradient(dl, bf16):
    x = draw(2, 129, 2, 64, 128, 1, seed=5, bf16=bf16)
    compare(run(dl, x, bf16, 1.0, init=False, d_final=False), x, bf16, 1.0, init=False, d_final=False)


@pytest.mark.parametrize("kind", ["no_decay", "reset", "minus_inf", "beta_zero", "beta_one", "same_key", "long_memory"])
@pytest.mark.parametrize("bf16", [True, False])
def test_gates_and_keys_at_their_ends(dl, kind, bf16):
    x = draw(2, 190, 2, 64, 128, 2, seed=11, bf16=bf16, relu_keys=kind == "same_key")
    r = np.random.default_rng(1)
    if kind == "no_decay":
        x["g"][:] = 0.0
    elif kind == "reset":        # a decay that forgets everything, at single tokens
        x["g"][r.uniform(size=x["g"].shape) < 0.05] = -300.0
    elif kind == "minus_inf":
        x["g"][:, :, 70] = -np.inf
        x["g"][:, 0, 64] = -np.inf
    elif kind == "beta_zero":
        x["beta"][r.uniform(size=x["beta"].shape) < 0.5] = 0.0
        x["beta"][0, 0] = 0.0
    elif kind == "beta_one":
        x["beta"][:] = 1.0
    elif kind == "same_key":     # strongly correlated keys
        x["g"][:] *= 0.01
    elif kind == "long_memory":
        x["g"][:] = -1e-4
        x["beta"][:] = 0.01
    out = run(dl, x, bf16, 0.4)
    with np.errstate(invalid="ignore"):
        compare(out, x, bf16, 0.4)


def test_step_matches_sequence_and_pool(dl):
    for bf16 in (True, False):
        for (b, H, P, N, G) in ((1, 4, 64, 128, 2), (5, 3, 40, 72, 1), (3, 2, 128, 256, 2), (2, 2, 4, 4, 1)):
            x = draw(b, 6, H, P, N, G, seed=b + H, bf16=bf16)
            d = dev(x, bf16)
            r = np.random.default_rng(2)
            pool = r.standard_normal((b + 4, H, P, N)).astype(np.float32)
            idx = r.permutation(b + 4)[:b].astype(np.int32)
            if b > 2:
                idx[1], idx[2] = -1, b + 4  # absent requests
            state, ref = torch.from_numpy(pool).cuda(), pool.astype(np.float64)
            for t in range(6):
                o = dl.delta_step(d["q"][:, t].contiguous(), d["k"][:, t].contiguous(), d["v"][:, t].contiguous(),
                                  d["g"][:, :, t].contiguous(), d["beta"][:, :, t].contiguous(), state, scale=0.6,
                                  state_index=torch.from_numpy(idx).cuda())
                ro = od.delta_step(x["q"][:, t], x["k"][:, t], x["v"][:, t], x["g"][:, :, t], x["beta"][:, :, t], 0.6, ref, idx)
                check(o, ro, BF16_BAR if bf16 else F32_BAR, "o", 1)
            check(state, ref, F32_BAR, "state", 1)
            if b > 2:
                assert torch.all(o[1] == 0) and torch.all(o[2] == 0)
            untouched = [i for i in range(b + 4) if i not in idx]
            assert torch.equal(state[untouched].cpu(), torch.from_numpy(pool[untouched]))


def test_prefill_then_steps(dl):
    # the chunked forward's state continues token by token
    x = draw(2, 150, 4, 64, 128, 2, seed=21)
    d = dev(x, True)
    cut = 133
    part = [d[k][:, :cut].contiguous() for k in ("q", "k", "v")] + [d[k][:, :, :cut].contiguous() for k in ("g", "beta")]
    o, state = dl.delta_forward(*part, scale=0.5, init_state=d["init"])
    outs = [o]
    for t in range(cut, 150):
        outs.append(dl.delta_step(d["q"][:, t].contiguous(), d["k"][:, t].contiguous(), d["v"][:, t].contiguous(),
                                  d["g"][:, :, t].contiguous(), d["beta"][:, :, t].contiguous(), state, scale=0.5)[:, None])
    ro, rS = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["init"])
    check(torch.cat(outs, 1), ro, BF16_BAR, "o", 2)
    check(state, rS, SPLIT_BAR, "state", 2)


def test_same_inputs_same_bits_and_other_streams(dl):
    x = draw(2, 300, 8, 64, 128, 2, seed=31)
    first = run(dl, x, True, 0.2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run(dl, x, True, 0.2)
    for k in first:
        assert torch.equal(first[k], second[k]), k


def test_backward_against_differences_of_the_forward(dl):
    # fp32: the gradient along a direction, against central differences of the GPU's own forward in fp32.
    # The loss is O(1) per term over ~1e4 terms; a step of 1e-2 leaves rounding ~1e-5 and curvature ~1e-3 relative.
    x = draw(1, 80, 2, 16, 32, 1, seed=41, bf16=False)
    d = dev(x, False)
    gr = dl.delta_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], scale=0.5, d_final_state=d["d_final"],
                           init_state=d["init"])
    gen = torch.Generator(device="cuda").manual_seed(0)

    def loss(e):
        o, S = dl.delta_forward(e["q"], e["k"], e["v"], e["g"], e["beta"], scale=0.5, init_state=e["init"])
        return float((o.double() * d["do"]).sum() + (S.double() * d["d_final"]).sum())

    for name, g in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("init", "d_init")):
        u = torch.randn(d[name].shape, generator=gen, device="cuda")
        u /= u.norm()
        h = 1e-2
        num = (loss(dict(d, **{name: d[name] + h * u})) - loss(dict(d, **{name: d[name] - h * u}))) / (2 * h)
        ana = float((gr[g].double() * u).sum())
        assert abs(num - ana) <= 1e-3 * float(gr[g].norm()) + 1e-3, (name, num, ana)


def test_clamped_valid_len_is_reported(dl):
    from state_space_model_mamba_gb300 import ssd
    x = draw(2, 20, 2, 64, 128, 1, seed=51)
    d = dev(x, True)
    vl = torch.tensor([25, -3], dtype=torch.int32, device="cuda")
    for simt in (False, True):
        with pytest.raises(ssd.SsdError, match="2 valid_len entries"):
            dl.delta_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], valid_len=vl, simt=simt, check_status=True)
        with pytest.raises(ssd.SsdError, match="2 valid_len entries"):
            dl.delta_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], valid_len=vl, simt=simt,
                              check_status=True)


def test_refusals(dl):
    x = dev(draw(1, 20, 4, 64, 128, 2, seed=61), True)
    a = dict(q=x["q"], k=x["k"], v=x["v"], g=x["g"], beta=x["beta"])
    for name, bad in (("q", x["q"].float()), ("k", x["k"][:, :-1]), ("g", x["g"].bfloat16()), ("beta", x["beta"][:, :2]),
                      ("q", x["q"].transpose(1, 2)), ("v", x["v"].half())):
        with pytest.raises((ValueError, TypeError)):
            dl.delta_forward(**dict(a, **{name: bad}))
    with pytest.raises(ValueError):
        dl.delta_forward(**a, init_state=x["init"].bfloat16())
    with pytest.raises(ValueError):
        dl.delta_forward(**a, valid_len=torch.tensor([20], device="cuda"))  # int64
    with pytest.raises(ValueError):
        dl.delta_backward(**a, do=x["do"].float())
    with pytest.raises(ValueError):
        dl.delta_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0].contiguous(), x["g"][:, :, 0], x["beta"][:, :, 0], x["init"])


def test_more_absent_tokens_than_32_bits_count(dl):
    """Token by token a block makes the absent tokens of its rows zero: 8 rows of 2^28 tokens and more."""
    import ctypes
    from state_space_model_mamba_gb300 import ssd
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB")
    L, valid, W = 2 ** 28 + 70, 5, 4
    x = draw(1, valid, 1, W, W, 1, seed=9, bf16=False)
    d = dev(x, False)

    def padded(t, axis):
        shape = list(t.shape)
        shape[axis] = L
        out = torch.zeros(shape, device="cuda")
        out.narrow(axis, 0, valid).copy_(t)
        return out

    q, k, v, do = (padded(d[n], 1) for n in ("q", "k", "v", "do"))
    g, beta = padded(d["g"], 2), padded(d["beta"], 2)
    vl = torch.tensor([valid], dtype=torch.int32, device="cuda")
    dims = dl.DeltaDims(1, L, 1, W, W, 1, 0, 0)
    nan = float("nan")
    stream = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(dl.workspace_bytes(dims, 0, True), dtype=torch.uint8, device="cuda")
    o, dv = torch.full_like(v, nan), torch.full_like(v, nan)
    five = [t.data_ptr() for t in (q, k, v, g, beta)]
    ssd._check(dl._lib().delta_forward(ctypes.byref(dims), 0, *five, 0.5, None, vl.data_ptr(), o.data_ptr(), None, ws.data_ptr(),
                                       ws.numel(), stream))
    ro, _ = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5)
    check(o[:, :valid], ro, F32_BAR, "o", 2)
    assert int(torch.count_nonzero(o[:, valid:])) == 0  # NaN counts
    del o
    dq, dk, dg, dbeta = torch.full_like(q, nan), torch.full_like(k, nan), torch.full_like(g, nan), torch.full_like(beta, nan)
    ssd._check(dl._lib().delta_backward(ctypes.byref(dims), 0, *five, 0.5, None, vl.data_ptr(), do.data_ptr(), None, dq.data_ptr(),
                                        dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), None, ws.data_ptr(),
                                        ws.numel(), stream))
    ref = od.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["do"])
    for name, t, axis in (("dq", dq, 1), ("dk", dk, 1), ("dv", dv, 1), ("dg", dg, 2), ("dbeta", dbeta, 2)):
        check(t.narrow(axis, 0, valid), ref[name], F32_BAR, name, 2)
        assert int(torch.count_nonzero(t.narrow(axis, valid, L - valid))) == 0, name


def strong_decay(L, zero_do, seed):
    """Heads that forget at one rate throughout."""
    x = draw(2, L, 4, 64, 128, 2, seed=seed)
    x["g"][:] = -np.array([6.0, 8.0, 10.0, 12.0], np.float32)[None, :, None]
    if zero_do:
        x["do"][:] = 0
    return x


@pytest.mark.parametrize("L", [64, 190])
def test_gate_gradients_under_strong_decay(dl, L):
    """A gradient of the final state alone: the last tokens' shares of dg are exp(6 .. 12) times those of the tokens
    before them.  Every head by its own norm; the bar is that of slices."""
    x = strong_decay(L, True, 71)
    out = run(dl, x, True, 0.4)
    ref = od.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.4, x["do"], x["d_final"], x["init"])
    for name in ("dg", "dbeta"):
        e = np.linalg.norm(out[name].double().cpu().numpy() - ref[name], axis=2) / np.linalg.norm(ref[name], axis=2)
        assert e.max() <= 4 * SPLIT_BAR, (name, e)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("L", [64, 190])
def test_gradients_under_strong_decay(dl, L, simt):
    """All that crosses a token is made small by its decay, and so is dg: what does not cross it must not be in the
    sum.  Every head by its own norm, not floored by those of others; the bars are those of slices."""
    x = strong_decay(L, False, 72)
    out = run(dl, x, True, 0.4, simt=simt)
    ref = od.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.4, x["do"], x["d_final"], x["init"])
    for name, axes, bar in (("dg", 2, SPLIT_BAR), ("dbeta", 2, SPLIT_BAR), ("dv", (1, 3), BF16_BAR), ("d_init", (2, 3), SPLIT_BAR)):
        e = np.linalg.norm(out[name].double().cpu().numpy() - ref[name], axis=axes) / np.linalg.norm(ref[name], axis=axes)
        assert e.max() <= 4 * bar, (name, e)


@pytest.mark.parametrize("shape", [(2, 300, 4, 64, 128, 4), (1, 450, 6, 128, 128, 2), (2, 200, 4, 64, 64, 1), (1, 333, 2, 96, 80, 2),
                                   (2, 130, 3, 64, 128, 1)])
def test_key_gradients_are_rounded_once(dl, shape):
    """dq, dk and dv in bf16: one rounding is 1.5e-3 to 1.7e-3 root-mean-square of values spread over a power of two
    or normal ones, and operands in two parts add nothing to it in quadrature: 2^-9."""
    x = draw(*shape, seed=80 + sum(shape))
    out = run(dl, x, True, 0.5)
    ref = od.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["do"], x["d_final"], x["init"])
    for name in ("dq", "dk", "dv"):
        check(out[name], ref[name], 2.0 ** -9, name, 2)


@pytest.mark.parametrize("shape", [(1, 333, 16, 128, 128, 8), (1, 257, 40, 64, 64, 8), (1, 190, 100, 64, 128, 100), (3, 150, 64, 64, 128, 8),
                                   (2, 200, 3, 96, 80, 1)])
def test_states_take_up_what_is_written_in_three_parts(dl, shape):
    """final_state and d_init.  What is added to a state is 2^-25 off; the products before that have operands in two
    parts (2^-17 at most, 2^-18.6 root-mean-square), of which the triangle's entries, some 0.2 of the diagonal, pass on
    a fifth each: X and Tt, and the solve behind Tt, 5e-7 each, decays of 2^-22.  In quadrature 9e-7; the bar is 1.5e-6."""
    x = draw(*shape, seed=90 + sum(shape))
    out = run(dl, x, True, 0.5)
    ref = od.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["do"], x["d_final"], x["init"])
    _, S = od.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.5, x["init"])
    for name, r in (("final", S), ("d_init", ref["d_init"])):
        e = np.linalg.norm(out[name].double().cpu().numpy() - r) / np.linalg.norm(r)
        assert e <= 1.5e-6, (name, e)


@pytest.mark.parametrize("shape, valid", [((2, 965, 39, 128, 8, 3), None), ((3, 970, 26, 96, 8, 13), [970, 100, 961])])
def test_halves_of_the_batch_with_two_slices_a_head(dl, shape, valid):
    """More chain slices than SMs over 16 chunks: each half's share of the workspace begins after whole heads of two slices."""
    x = draw(*shape, seed=sum(shape))
    compare(run(dl, x, True, 0.3, valid=valid), x, True, 0.3, valid=valid)
