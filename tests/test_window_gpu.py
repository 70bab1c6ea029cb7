"""GPU parity of window attention (include/window.h), through the C ABI, against the
fp64 oracle (oracle/window.py).

Bars, as normwise relative errors of whole outputs (a rounding is at most eps / 2 of a value, 0.29 eps / sqrt(2) ..
0.41 eps / 2 root-mean-square: 1.7e-3 at most in bf16):
  * fp32 storage: dot products of at most 128 terms, scores of a few units, sums over at most some hundred
    keys, a handful of roundings each (2^-24): 1e-5;
  * bf16 storage, o and dv: the output's rounding (1.7e-3) and the probabilities' (1.7e-3), in quadrature 2.4e-3: 2^-8;
  * bf16 storage, dq and dk: the output's, that of the scores' gradients and that of o in do.o, which enters
    with p (do.v - do.o) where |o| <= |v|: 2.9e-3: 2^-8;
  * lse in either: sums in fp32, exact products: 1e-5.
Slices along the leading axes are held to four times the bar, their norms floored at a tenth of the
tensor's RMS slice norm: a single row's roundings are not averaged.  Rows of dq and dk (and so the norm of all of
them, by the norm of the rows' bounds) are allowed on top what the rounding of do.o moves them by
(oracle/window.py, rounding_of_o): where p all but sits on one key, do.v - do.o cancels and that does not.  In bf16 it is o's, 2^-8 of every term; in fp32 the sum's, P roundings of 2^-24."""
import numpy as np
import pytest

from oracle import window as ow

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32_BAR, BF16_BAR = 1e-5, 2.0 ** -8


@pytest.fixture(scope="module")
def wd():
    from state_space_model_mamba_gb300 import window
    return window


def store(a, bf16):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    return (t.bfloat16().float() if bf16 else t).numpy()


def draw(b, L, H, G, P, seed, bf16=True):
    r = np.random.default_rng(seed)
    common = 0.5 * r.standard_normal(P)
    return dict(q=store(r.standard_normal((b, L, H, P)) + common, bf16), k=store(r.standard_normal((b, L, G, P)) + common, bf16),
                v=store(r.standard_normal((b, L, G, P)), bf16), do=store(r.standard_normal((b, L, H, P)), bf16))


def dev(a, bf16):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.bfloat16 if bf16 else torch.float32)


def ints(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def check(got, ref, bar, what, axes, off=0.0):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    d, n = got - ref, np.linalg.norm(ref)
    whole = max(np.linalg.norm(d) - np.linalg.norm(off), 0.0) / (n if n else 1.0)
    assert whole <= bar, f"{what}: {whole:.3e} > {bar:.3e}"
    m = int(np.prod(ref.shape[:axes]))
    rn = np.linalg.norm(ref.reshape(m, -1), axis=1)
    floor = max(0.1 * np.sqrt(np.mean(rn ** 2)), 1e-30)
    rows = np.maximum(np.linalg.norm(d.reshape(m, -1), axis=1) - np.ravel(off), 0.0)
    worst = np.max(rows / np.maximum(rn, floor))
    assert worst <= 4 * bar, f"{what}, worst slice: {worst:.3e} > {4 * bar:.3e}"


def run(wd, x, W, sinks, bf16, scale=None, valid=None, simt=False, backward=True):
    d = {k: dev(a, bf16) for k, a in x.items()}
    vl = ints(valid)
    o, lse = wd.window_forward(d["q"], d["k"], d["v"], W, sinks, scale=scale, valid_len=vl, simt=simt)
    out = dict(o=o, lse=lse)
    if backward:
        out.update(wd.window_backward(d["q"], d["k"], d["v"], o, lse, d["do"], W, sinks, scale=scale, valid_len=vl, simt=simt))
    torch.cuda.synchronize()
    return out


def compare(out, x, W, sinks, bf16, scale=None, valid=None):
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    o, lse = ow.window_forward(x["q"], x["k"], x["v"], W, sinks, scale, valid)
    ref = dict(o=o, lse=lse)
    if "dq" in out:
        ref.update(ow.window_backward(x["q"], x["k"], x["v"], x["do"], W, sinks, scale, valid))
    off = ow.rounding_of_o(x["q"], x["k"], x["v"], x["do"], W, sinks, scale, valid) if "dq" in out else {}
    if not bf16:
        off = {name: a * x["q"].shape[-1] * 2.0 ** -16 for name, a in off.items()}
    for name, r in ref.items():
        check(out[name], r, F32_BAR if not bf16 or name == "lse" else BF16_BAR, name, 2 if name == "lse" else 3, off.get(name, 0.0))


# one token; tile edges; ragged tails; windows inside and across tiles, wider than the row, of one; sinks inside the
# window, in front of it, more than a tile; shared heads that do and do not divide a tile; padded widths
SHAPES = [(1, 2, 1, 1, 64, 4, 0), (2, 63, 2, 2, 64, 17, 3), (1, 128, 4, 2, 128, 128, 0), (2, 129, 4, 1, 64, 64, 1),
          (1, 300, 2, 2, 64, 100, 130), (1, 260, 5, 1, 128, 33, 4), (1, 200, 6, 2, 96, 1000, 0), (2, 150, 3, 1, 8, 40, 16),
          (1, 513, 1, 1, 64, 129, 4), (1, 700, 2, 1, 128, 256, 128), (1, 400, 8, 1, 80, 2, 5), (1, 70, 33, 1, 64, 20, 2),
          (1, 140, 128, 1, 64, 50, 4), (1, 90, 130, 1, 64, 50, 4)]


@pytest.mark.parametrize("b,L,H,G,P,W,sinks", SHAPES)
def test_simt_bf16(wd, b, L, H, G, P, W, sinks):
    x = draw(b, L, H, G, P, L + W)
    compare(run(wd, x, W, sinks, True, simt=True), x, W, sinks, True)


@pytest.mark.parametrize("b,L,H,G,P,W,sinks", SHAPES)
def test_bf16(wd, b, L, H, G, P, W, sinks):
    x = draw(b, L, H, G, P, L + W)
    compare(run(wd, x, W, sinks, True), x, W, sinks, True)


@pytest.mark.parametrize("b,L,H,G,P,W,sinks", SHAPES[:9] + [(2, 33, 3, 1, 4, 7, 2), (1, 40, 2, 2, 36, 9, 0), (1, 50, 2, 1, 124, 9, 3)])
def test_f32(wd, b, L, H, G, P, W, sinks):
    x = draw(b, L, H, G, P, L + W, bf16=False)
    compare(run(wd, x, W, sinks, False), x, W, sinks, False)


@pytest.mark.parametrize("b,L,H,G,P,W,sinks", [(2, 650, 8, 8, 20, 100, 0), (1, 700, 12, 2, 64, 33, 3), (3, 333, 16, 16, 128, 50, 0),
                                               (2, 900, 8, 4, 36, 20, 5)])
def test_f32_blocks_on_every_sm(wd, b, L, H, G, P, W, sinks):
    """Enough blocks of 32 rows for the form with four rows a warp; narrow heads; sinks far behind the window."""
    x = draw(b, L, H, G, P, L + P, False)
    valid = [L] + [L // 2 + 7 * i for i in range(b - 1)]
    compare(run(wd, x, W, sinks, False, valid=valid), x, W, sinks, False, valid=valid)


@pytest.mark.parametrize("bf16", [False, True])
def test_a_token_that_sees_itself_alone(wd, bf16):
    """window 1 without sinks: o = v exactly, lse the score, gradients of q and k only what do.o loses to o's rounding."""
    x = draw(2, 40, 4, 2, 64, 3, bf16)
    out = run(wd, x, 1, 0, bf16)
    assert torch.equal(out["o"], dev(np.repeat(x["v"], 2, axis=2), bf16))
    s = np.einsum("blhp,blhp->bhl", x["q"].astype(float), np.repeat(x["k"], 2, axis=2).astype(float)) / 8
    assert np.abs(out["lse"].double().cpu().numpy() - s).max() < 1e-5
    # o is v exactly, so do.o is do.v up to fp32 sums of 64 terms of size 1
    assert out["dq"].float().abs().max() < 64 * 2 ** -22 and out["dk"].float().abs().max() < 64 * 2 ** -22
    ref = x["do"].reshape(2, 40, 2, 2, 64).sum(3)
    check(out["dv"], ref.astype(np.float64), BF16_BAR if bf16 else F32_BAR, "dv", 2)


@pytest.mark.parametrize("bf16,simt", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("W,sinks", [(50, 4), (500, 0), (9, 150)])
def test_absent_tokens(wd, bf16, simt, W, sinks):
    """Rows of every length (none, one, tile edges, all), NaN and infinities in what is absent, lengths out of range."""
    valid = [0, 1, 128, 130, 300, 255]
    x = draw(6, 300, 4, 2, 64, 11, bf16)
    y = {k: a.copy() for k, a in x.items()}
    for i, V in enumerate(valid):
        for j, name in enumerate(y):
            y[name][i, V:] = [np.nan, np.inf, -np.inf, np.nan][(i + j) % 4]
    out = run(wd, y, W, sinks, bf16, valid=valid, simt=simt)
    compare(out, x, W, sinks, bf16, valid=valid)
    for i, V in enumerate(valid):
        assert not out["lse"][i, :, V:].any()
        for name in ("o", "dq", "dk", "dv"):
            assert not out[name][i, V:].any()
    from state_space_model_mamba_gb300 import ssd
    d = {k: dev(a, bf16) for k, a in x.items()}
    o, _ = wd.window_forward(d["q"], d["k"], d["v"], W, sinks, valid_len=ints([-3, 1, 128, 130, 999, 255]), simt=simt)
    assert torch.equal(o, out["o"])
    with pytest.raises(ssd.SsdError, match="2"):
        wd.window_forward(d["q"], d["k"], d["v"], W, sinks, valid_len=ints([-3, 1, 128, 130, 999, 255]), simt=simt, check_status=True)


@pytest.mark.parametrize("bf16,simt", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("size", [30.0, -30.0, 1e-3])
def test_scores_of_every_size(wd, bf16, simt, size):
    """Scales that make rows of a single key, of all keys alike, and negative ones; scores of some thousands.
    Errors of a score are 2^-24 of it times its sums' length, up to some 1e-3 at scores of thousands, and so are those of p."""
    x = draw(1, 200, 2, 1, 64, 12, bf16)
    out = run(wd, x, 70, 3, bf16, scale=size, simt=simt, backward=False)
    o, lse = ow.window_forward(x["q"], x["k"], x["v"], 70, 3, size)
    s = max(1.0, np.abs(lse).max())
    check(out["lse"], lse, F32_BAR, "lse", 2)
    check(out["o"], o, (BF16_BAR if bf16 else F32_BAR) + 8 * s * 2.0 ** -23, "o", 3)


@pytest.mark.parametrize("bf16,simt", [(False, False), (True, False), (True, True)])
def test_same_bits_every_time_and_in_a_graph(wd, bf16, simt):
    x = draw(2, 1100, 8, 2, 64, 13, bf16)
    d = {k: dev(a, bf16) for k, a in x.items()}
    vl = ints([1100, 900])

    def step():
        o, lse = wd.window_forward(d["q"], d["k"], d["v"], 200, 4, valid_len=vl, simt=simt)
        g = wd.window_backward(d["q"], d["k"], d["v"], o, lse, d["do"], 200, 4, valid_len=vl, simt=simt)
        return [o, lse, g["dq"], g["dk"], g["dv"]]

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = step()
    for t in third:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_no_lse_and_default_scale(wd):
    x = draw(1, 50, 2, 2, 64, 14)
    d = {k: dev(a, True) for k, a in x.items()}
    o, lse = wd.window_forward(d["q"], d["k"], d["v"], 20, return_lse=False)
    assert lse is None and torch.equal(o, wd.window_forward(d["q"], d["k"], d["v"], 20, 0, scale=0.125)[0])


def test_guard_regions(wd):
    """Outputs between guard values, through the C ABI: nothing is written outside them."""
    import ctypes
    from state_space_model_mamba_gb300 import ssd
    for bf16, (b, L, H, G, P, W, sinks) in ((True, (2, 131, 5, 1, 72, 40, 3)), (False, (2, 37, 3, 1, 20, 9, 3))):
        x = draw(b, L, H, G, P, 15, bf16)
        d = {k: dev(a, bf16) for k, a in x.items()}
        T, code = (torch.bfloat16, 1) if bf16 else (torch.float32, 0)
        dims = wd.WindowDims(b, L, H, P, G, W, sinks, 0, 0)
        pad = 4096
        n = dict(o=b * L * H * P, lse=b * H * L, dq=b * L * H * P, dk=b * L * G * P, dv=b * L * G * P,
                 fw=wd.workspace_bytes(dims, code, False), bw=wd.workspace_bytes(dims, code, True))
        t = {k: torch.full((m + 2 * pad,), 77.0, device="cuda", dtype=torch.float32 if k == "lse" else
                           (torch.uint8 if k in ("fw", "bw") else T)) for k, m in n.items()}
        at = {k: a.data_ptr() + pad * a.element_size() for k, a in t.items()}
        lib, s = wd._lib(), torch.cuda.current_stream().cuda_stream
        ssd._check(lib.window_forward(ctypes.byref(dims), code, d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), 0.1, None,
                                      at["o"], at["lse"], at["fw"], n["fw"], s))
        ssd._check(lib.window_backward(ctypes.byref(dims), code, d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), at["o"],
                                       at["lse"], d["do"].data_ptr(), 0.1, None, at["dq"], at["dk"], at["dv"], at["bw"], n["bw"], s))
        torch.cuda.synchronize()
        for k, a in t.items():
            assert torch.all(a[:pad].float() == 77) and torch.all(a[-pad:].float() == 77), k
        o, lse = wd.window_forward(d["q"], d["k"], d["v"], W, sinks, scale=0.1)
        assert torch.equal(t["o"][pad:-pad].view_as(o), o) and torch.equal(t["lse"][pad:-pad].view_as(lse), lse)


# ------------------------------------------------------------------ the ring
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("b,L,G,P,W,sinks", [(3, 40, 2, 64, 16, 4), (2, 5, 1, 12, 16, 4), (2, 300, 3, 20, 7, 0), (1, 1, 1, 4, 1, 0),
                                             (3, 129, 2, 128, 64, 70)])
def test_fill(wd, b, L, G, P, W, sinks, bf16):
    x = draw(b, L, G, G, P, 16, bf16)
    k, v = dev(x["k"], bf16), dev(x["v"], bf16)
    for valid, index in ((None, None), ([max(1, L // 2)] + [L] * (b - 1), list(range(b, 0, -1))), ([0] * b, None),
                         (None, [-1] + list(range(b + 1, 2, -1))[:b - 1])):
        shape = (b + 2, sinks + W, G, P)
        kc, vc = torch.full(shape, 3.0, device="cuda", dtype=k.dtype), torch.full(shape, 5.0, device="cuda", dtype=k.dtype)
        wd.window_fill(k, v, kc, vc, W, sinks, valid_len=ints(valid), cache_index=ints(index))
        for cache, src, was in ((kc, x["k"], 3.0), (vc, x["v"], 5.0)):
            ref = ow.window_fill(src, np.full(shape, was, np.float32), W, sinks, valid, index)
            assert np.array_equal(cache.float().cpu().numpy(), ref)


STEPS = [(3, 4, 2, 64, 16, 4), (1, 40, 8, 128, 300, 4), (2, 1, 1, 64, 1, 0), (5, 16, 1, 96, 50, 0), (2, 33, 1, 80, 40, 2),
         (4, 8, 8, 8, 9, 3), (2, 6, 2, 40, 700, 130), (200, 2, 2, 64, 33, 1), (1, 5, 1, 128, 2500, 16)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("b,H,G,P,W,sinks", STEPS)
def test_step(wd, b, H, G, P, W, sinks, bf16):
    """Positions from the first token to far past the ring's end; what is not written yet holds NaN."""
    x = draw(b, 1, H, G, P, 17, bf16)
    r = np.random.default_rng(18)
    n = sinks + W
    pos = np.array([[0, 1, sinks, n - 1, n, 3 * n + 1, 2 ** 31 - 1, max(0, n - 2)][i % 8] for i in range(b)])[::-1].copy()
    index = r.permutation(b + 3)[:b]
    kc, vc = (store(r.standard_normal((b + 3, n, G, P)), bf16) for _ in range(2))
    for i in range(b):
        kc[index[i], pos[i]:] = np.nan
        vc[index[i], pos[i]:] = np.nan
    if b > 2:
        index[1] = -1 if b % 2 else b + 3
        pos[2] = -1
    dk, dv = dev(kc, bf16), dev(vc, bf16)
    q, k, v = (dev(x[name][:, 0], bf16) for name in "qkv")
    o = wd.window_step(q, k, v, dk, dv, ints(pos.tolist()), W, sinks, cache_index=ints(index.tolist()))
    ro, rk, rv = ow.window_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], kc, vc, pos, W, sinks, P ** -0.5, index)
    check(o, ro, BF16_BAR if bf16 else F32_BAR, "o", 2)
    assert np.array_equal(dk.double().cpu().numpy(), rk, equal_nan=True)
    assert np.array_equal(dv.double().cpu().numpy(), rv, equal_nan=True)
    if b > 2:
        assert not o[1].any() and not o[2].any()


def test_step_simt_width_and_slots_in_order(wd):
    """bf16 rows that are no multiple of 16 bytes; slots taken in order."""
    x = draw(2, 1, 3, 1, 20, 19)
    r = np.random.default_rng(20)
    kc, vc = (store(r.standard_normal((2, 30, 1, 20)), True) for _ in range(2))
    dk, dv = dev(kc, True), dev(vc, True)
    o = wd.window_step(*(dev(x[n][:, 0], True) for n in "qkv"), dk, dv, ints([5, 100]), 28, 2)
    ro, rk, rv = ow.window_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], kc, vc, [5, 100], 28, 2, 20 ** -0.5)
    check(o, ro, BF16_BAR, "o", 2)
    assert np.array_equal(dk.double().cpu().numpy(), rk) and np.array_equal(dv.double().cpu().numpy(), rv)


def test_cache_offsets_past_32_bits(wd):
    """The last slots of a ring of more than 2^32 bytes and 2^31 elements, against a ring of their own."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    slots, W, G, P = 1100, 16380, 1, 128
    kc, vc = (torch.empty(slots, W + 4, G, P, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    x = draw(2, 400, 4, G, P, 21)
    k, v = dev(x["k"], True), dev(x["v"], True)
    index = ints([slots - 1, slots - 2])
    sk, sv = (torch.empty(2, W + 4, G, P, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    wd.window_fill(k, v, kc, vc, W, 4, cache_index=index)
    wd.window_fill(k, v, sk, sv, W, 4, cache_index=ints([1, 0]))
    q, k1, v1 = (dev(x[n][:, 7], True) for n in "qkv")
    a = wd.window_step(q, k1, v1, kc, vc, ints([400, 400]), W, 4, cache_index=index)
    b = wd.window_step(q, k1, v1, sk, sv, ints([400, 400]), W, 4, cache_index=ints([1, 0]))
    assert torch.equal(a, b) and torch.equal(kc[-2:, :401], sk[:, :401]) and torch.equal(vc[-2:, :401], sv[:, :401])


@pytest.mark.parametrize("bf16", [False, True])
def test_prefill_then_steps_are_the_sequence(wd, bf16):
    """The operators together: prompts of different lengths, their rings, then captured steps, against whole sequences."""
    b, L, H, G, P, W, sinks, more = 3, 150, 8, 2, 64, 48, 3, 20
    x = draw(b, L, H, G, P, 22, bf16)
    lengths = [130, 1, 60]
    ref, _ = ow.window_forward(x["q"], x["k"], x["v"], W, sinks, P ** -0.5)
    d = {k: dev(a, bf16) for k, a in x.items()}
    vl, index = ints(lengths), ints([4, 0, 3])
    kc, vc = (torch.full((5, sinks + W, G, P), float("nan"), device="cuda", dtype=d["q"].dtype) for _ in range(2))
    o, _ = wd.window_forward(d["q"], d["k"], d["v"], W, sinks, valid_len=vl, return_lse=False)
    wd.window_fill(d["k"], d["v"], kc, vc, W, sinks, valid_len=vl, cache_index=index)
    bar = BF16_BAR if bf16 else F32_BAR
    for i, V in enumerate(lengths):
        check(o[i, :V], ref[i, :V], bar, "prompt", 2)
    rows, at = torch.arange(b, device="cuda"), ints(lengths)
    q, k, v = (d[n][rows, at.long()].contiguous() for n in "qkv")
    pos = at.clone()
    saved = kc.clone(), vc.clone()
    graph = torch.cuda.CUDAGraph()
    wd.window_step(q, k, v, kc, vc, pos, W, sinks, cache_index=index)
    with torch.cuda.graph(graph):
        got = wd.window_step(q, k, v, kc, vc, pos, W, sinks, cache_index=index)
    kc.copy_(saved[0]), vc.copy_(saved[1])
    for t in range(more):
        now = at + t
        for buf, n in ((q, "q"), (k, "k"), (v, "v")):
            buf.copy_(d[n][rows, now.long()])
        pos.copy_(now)
        graph.replay()
        check(got, ref[np.arange(b), np.array(lengths) + t], bar, f"token {t}", 2)
    assert torch.isnan(kc[1].float()).all() and torch.isnan(vc[2].float()).all()


def test_refusals(wd):
    from state_space_model_mamba_gb300 import ssd
    x = draw(2, 8, 4, 2, 64, 23)
    d = {k: dev(a, True) for k, a in x.items()}
    q, k, v = d["q"], d["k"], d["v"]
    for bad in ((q.float(), k, v), (q, k, v[:, :4]), (q[:, :, :3].contiguous(), k, v), (q.transpose(0, 1), k, v),
                (q, k.transpose(0, 1), v.transpose(0, 1)), (q[..., :32].contiguous(), k, v), (q[0], k, v)):
        with pytest.raises((ValueError, TypeError)):
            wd.window_forward(*bad, 4)
    with pytest.raises(TypeError):
        wd.window_forward(q.half(), k.half(), v.half(), 4)
    for W, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(ssd.SsdError, match="INVALID"):
            wd.window_forward(q, k, v, W, sinks)
    with pytest.raises(ssd.SsdError, match="UNSUPPORTED"):
        wd.window_forward(*(torch.zeros(1, 4, 1, 12, device="cuda", dtype=torch.bfloat16) for _ in range(3)), 4)
    with pytest.raises(ValueError, match="valid_len"):
        wd.window_forward(q, k, v, 4, valid_len=torch.tensor([8, 8], device="cuda"))
    o, lse = wd.window_forward(q, k, v, 4)
    for bad in ((o.float(), lse, d["do"]), (o, lse[:, :2], d["do"]), (o, lse, d["do"][:1])):
        with pytest.raises(ValueError):
            wd.window_backward(q, k, v, *bad, 4)
    kc = torch.zeros(3, 6, 2, 64, device="cuda", dtype=torch.bfloat16)
    for W, sinks, c, index in ((4, 1, kc, None), (4, 2, kc.float(), None), (4, 2, kc[0], None), (4, 2, kc, [0]), (4, 2, kc[:, :, :1], None)):
        with pytest.raises(ValueError):
            wd.window_fill(k, v, c, c, W, sinks, cache_index=ints(index))
        with pytest.raises(ValueError):
            wd.window_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), c, c, ints([0, 0]), W, sinks,
                           cache_index=ints(index))
    with pytest.raises(ssd.SsdError, match="slots"):
        wd.window_fill(k, v, kc[:1], kc[:1], 4, 2)
    with pytest.raises(ValueError, match="position"):
        wd.window_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), kc, kc.clone(), ints([0]), 4, 2)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("b,L,H,G,P,W,sinks", [(1, 300, 2, 1, 64, 20, 280), (2, 257, 4, 2, 128, 1, 1000), (1, 1500, 2, 2, 64, 30, 900),
                                               (1, 300, 2, 1, 64, 20, 279), (1, 2700, 1, 1, 8, 40, 300)])
def test_many_sinks(wd, b, L, H, G, P, W, sinks, simt):
    """Sinks that with the window cover the row (plain causal attention), all but cover it, take many tiles."""
    x = draw(b, L, H, G, P, L + sinks)
    valid = [L - 3 * i for i in range(b)]
    compare(run(wd, x, W, sinks, True, valid=valid, simt=simt), x, W, sinks, True, valid=valid)


@pytest.mark.parametrize("H,G,P", [(2, 2, 64), (4, 1, 128)])
@pytest.mark.parametrize("rise", [0.02, 0.3, -0.3, 8.0])
def test_scores_that_rise_and_fall_along_the_row(wd, H, G, P, rise):
    """Each tile's scores lie above (below) those of the tiles before, so that the softmax's reference has to move (stays) from tile
    to tile.  Tolerances as for scores of every size: a score is off by its length's sum times 2^-24 of it."""
    L, W, sinks = 700, 400, 3
    x = draw(1, L, H, G, P, 21)
    u = np.zeros(P, np.float32)
    u[0] = 1.0
    ramp = (np.arange(L, dtype=np.float32) - L / 2) * rise
    x["q"] = store(0.3 * x["q"] + u, True)
    x["k"] = store(0.3 * x["k"] + ramp[None, :, None, None] * u, True)
    out = run(wd, x, W, sinks, True, scale=1.0, backward=False)
    o, lse = ow.window_forward(x["q"], x["k"], x["v"], W, sinks, 1.0)
    s = max(1.0, np.abs(lse).max())
    check(out["lse"], lse, F32_BAR, "lse", 2)
    check(out["o"], o, BF16_BAR + 8 * s * 2.0 ** -23, "o", 3)
