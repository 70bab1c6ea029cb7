"""The operators measured here: attention with a sliding window and sinks (prefill
with its ring cache, training step, one-token step), the mixers' exit norm (group norm
per token with a gate, forward and backward) and the scan's one-token step.

``run`` computes them either in a plain form (elementary torch operations in
fp32, rounded once at the end) or, with ``own`` set, through this package.
``exact`` is the same in 64 bits from the definitions:

  window attention, query head h of key group g = h / (H / G), token t of V present ones:
      o_t = sum_s p_ts v_s,  p_t = softmax over s of scale q_t . k_s,
      s visible where s <= t and (t - s < window or s < sinks);  lse_t = log sum_s exp(scale q_t . k_s)
      (tokens at or past valid_len are absent: outputs and gradients are 0)
  ring cache of sinks + window entries a slot: token t lies at t where t < sinks, else at
      sinks + (t - sinks) mod window
  exit norm, per token and group of channels:  u = x, or x act(gate) with gate_first;
      n = (u - mean) / sqrt(mean((u - mean)^2) + eps), without centring u / sqrt(mean(u^2) + eps);
      y = n weight + bias, then times act(gate), or act(y) without a gate
  scan step:  S = exp(dt A) S + dt x (x) B,  y = S C + D x
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 512  # query tokens per block of the plain form


# ------------------------------------------------------------------ the cases
def _attn(name, op, b, L, H, G, P, window, sinks, dtype="bf16", ragged=False):
    return dict(name=name, op=op, b=b, L=L, H=H, G=G, P=P, window=window, sinks=sinks, dtype=dtype, ragged=ragged)


def listed():
    return [
        # a short prompt of one request into its ring: latency counts
        _attn("prefill_prompt", "prefill", 1, 333, 16, 8, 128, 256, 4),
        # a prefill batch of padded prompts of different lengths (the grouped, padded workload's shape)
        _attn("prefill_padded", "prefill", 8, 4096, 64, 8, 64, 1024, 4, ragged=True),
        # one document of 131072 tokens (the long-sequence workload's length and heads)
        _attn("prefill_long", "prefill", 1, 131072, 32, 8, 128, 1024, 4),
        # fp32 gradient-check run at a small size: forward and backward
        _attn("train_f32", "train", 2, 129, 4, 2, 32, 48, 2, dtype="f32"),
        # training step of the 130M layer: heads of 64, a short window without sinks
        _attn("train_130m", "train", 4, 2048, 24, 24, 64, 512, 0),
        # training step of the 2.7B layer: its 5120 channels as 40 heads of 128, keys shared by five heads
        _attn("train_2p7b", "train", 2, 8192, 40, 8, 128, 2048, 4),
        # one decoded token of one request with a full ring, and of a batch of old and young requests from a larger pool
        dict(name="step_one", op="step", b=1, H=40, G=8, P=128, window=2048, sinks=4, slots=4, young=False, dtype="bf16"),
        dict(name="step_batch", op="step", b=192, H=40, G=8, P=128, window=1024, sinks=4, slots=256, young=True, dtype="bf16"),
        # the mixers' exit: a decode batch (gate first, no centring: the scan layer's form), and a training step of the
        # 2.7B layer's tokens, each head of 64 normed and then gated
        dict(name="exit_decode", op="exit", rows=24, D=5120, groups=8, dtype="bf16", gate="first", center=False, bias=False,
             act="silu"),
        dict(name="exit_train", op="exit_train", rows=16384, D=5120, groups=80, dtype="bf16", gate="after", center=True, bias=True,
             act="silu"),
        # the scan's decoded token: one request, and a batch drawn from a larger pool of states
        dict(name="scan_step_one", op="scan_step", b=1, H=80, P=64, N=128, G=1, slots=4, dtype="bf16"),
        dict(name="scan_step_batch", op="scan_step", b=192, H=80, P=64, N=128, G=1, slots=256, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "step", "exit", "exit_train", "scan_step"])
    if op in ("prefill", "train"):
        if rng.random() < 0.8:
            P, G, dtype, most = rng.choice([64, 64, 128, 128, 96, 80]), _log(rng, 1, 16), "bf16", 2e12
            H, b = G * rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 1, 2, 3, 4])
        else:
            P, G, dtype, most = 4 * rng.randint(2, 16), rng.choice([1, 2]), "f32", 1e9
            H, b = G * rng.choice([1, 2, 3]), rng.choice([1, 2])
        # a token that sees itself alone has no gradient to measure: training windows and rows start at 16
        window, sinks = _log(rng, 1 if op == "prefill" else 16, 4096), rng.choice([0, 1, 4, 4, 16, 128])
        # the work of all tokens and heads stays below the largest listed case's
        L = _log(rng, 1 if op == "prefill" else 16, min(8192 if op == "train" else 65536, int(most / (14 * b * H * P * (window + sinks + 512))) + 17))
        return dict(op=op, b=b, L=L, H=H, G=G, P=P, window=window, sinks=sinks, dtype=dtype,
                    ragged=rng.random() < 0.4)
    if op == "step":
        G, b = _log(rng, 1, 8), _log(rng, 1, 192)
        return dict(op=op, b=b, H=G * rng.choice([1, 2, 4, 5, 8]), G=G, P=rng.choice([64, 64, 128, 96, 40]),
                    window=_log(rng, 1, 1024 if b > 16 else 8192), sinks=rng.choice([0, 1, 4, 4, 16, 128]),
                    slots=b + rng.randint(0, 32), young=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "scan_step":
        H, b = 4 * _log(rng, 1, 20), _log(rng, 1, 192)
        return dict(op=op, b=b, H=H, P=rng.choice([64, 64, 128, 40]), N=rng.choice([128, 128, 64, 16]),
                    G=H // rng.choice([1, 2, 4, H]), slots=b + rng.randint(0, 64), dtype=rng.choice(["bf16", "bf16", "f32"]))
    width = rng.choice([64, 64, 128, 128, 96, 256, 512, 8 * rng.randint(1, 40), rng.randint(3, 700)])
    groups = _log(rng, 1, min(80, 16384 // width))
    return dict(op=op, rows=_log(rng, 1, 60_000_000 // (width * groups)), D=width * groups, groups=groups,
                dtype=rng.choice(["bf16", "bf16", "f32"]), gate=rng.choice(["first", "after", "after", "none"]),
                center=rng.random() < 0.5, bias=rng.random() < 0.5, act=rng.choice(["silu", "silu", "sigmoid"]))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen, T, op = torch.Generator(device=DEV).manual_seed(seed), TYPES[case["dtype"]], case["op"]

    def randn(*s):
        return torch.randn(*s, generator=gen, device=DEV)

    s = dict(op=op)
    if op in ("exit", "exit_train"):
        R, D = case["rows"], case["D"]
        s.update({k: case[k] for k in ("groups", "center", "act")}, eps=1e-5, first=case["gate"] == "first")
        s["x"] = (0.7 * randn(R, D) + 0.2 * randn(1, D)).to(T)  # a mixer's output: channels have means of their own
        s["gate"] = randn(R, D).to(T) if case["gate"] != "none" else None
        s["weight"] = 1.0 + 0.1 * randn(D)
        s["bias"] = 0.1 * randn(D) if case["bias"] else None
        if op == "exit_train":
            s["dy"] = randn(R, D).to(T)
        return s
    b, H, G, P = case["b"], case["H"], case["G"], case["P"]
    if op == "scan_step":
        N = case["N"]
        s["x"], s["B"], s["C"] = randn(b, H, P).to(T), randn(b, G, N).to(T), randn(b, G, N).to(T)
        s["dt"] = torch.nn.functional.softplus(randn(b, H) - 3.0)
        s["A"] = -torch.exp(math.log(16.0) * torch.rand(H, generator=gen, device=DEV))
        s["D"] = 1.0 + 0.1 * randn(H)
        s["state"] = 0.3 * randn(case["slots"], H, P, N)
        s["index"] = torch.randperm(case["slots"], generator=gen, device=DEV)[:b].to(torch.int32)
        return s
    s["window"], s["sinks"], s["scale"] = case["window"], case["sinks"], P ** -0.5
    lead = (b,) if op == "step" else (b, case["L"])
    # queries and keys of norm sqrt(P), with a share in common, so that softmax rows are neither flat nor single
    s["q"] = (randn(*lead, H, P) + 0.5 * randn(1, 1, P)).to(T)
    s["k"] = (randn(*lead, G, P) + 0.5 * randn(1, 1, P)).to(T)
    s["v"] = randn(*lead, G, P).to(T)
    entries = case["sinks"] + case["window"]
    if op == "step":
        s["k_cache"], s["v_cache"] = randn(case["slots"], entries, G, P).to(T), randn(case["slots"], entries, G, P).to(T)
        lo, hi = (0, 2 * entries) if case["young"] else (entries, 9 * entries)
        s["position"] = torch.randint(lo, hi, (b,), generator=gen, device=DEV).to(torch.int32)
        s["index"] = torch.randperm(case["slots"], generator=gen, device=DEV)[:b].to(torch.int32)
        return s
    s["valid_len"] = None
    if case["ragged"]:
        L = case["L"]
        s["valid_len"] = torch.randint(min(L, max(1, L // 4)), L + 1, (b,), generator=gen, device=DEV).to(torch.int32)
    if op == "train":
        s["do"] = randn(b, case["L"], H, P).to(T)
    else:
        s["k_cache"], s["v_cache"] = (torch.zeros(b + 1, entries, G, P, dtype=T, device=DEV) for _ in range(2))
        s["index"] = torch.randperm(b + 1, generator=gen, device=DEV)[:b].to(torch.int32)
    return s


# ------------------------------------------------------------------ plain forms
def _present(s, b, L):
    if s["valid_len"] is None:
        return torch.ones(b, L, dtype=torch.bool, device=DEV)
    return torch.arange(L, device=DEV)[None, :] < s["valid_len"].clamp(0, L)[:, None]


def _plain_blocks(s, each):
    """Calls each(t0, t1, keys' slices, probabilities, log sums) for every block of queries; the keys a block sees
    are the sinks in front of its window and the tokens from there on, as [b, G, R, queries, keys]."""
    b, L, H, P = s["q"].shape
    G, W = s["k"].shape[2], s["window"]
    for t0 in range(0, L, BLOCK):
        t1 = min(L, t0 + BLOCK)
        lo = max(0, t0 - W + 1)
        parts = [slice(0, min(s["sinks"], lo)), slice(lo, t1)]
        keys = torch.cat([torch.arange(x.start, x.stop, device=DEV) for x in parts])
        t = torch.arange(t0, t1, device=DEV)[:, None]
        seen = (keys[None, :] <= t) & ((t - keys[None, :] < W) | (keys[None, :] < s["sinks"]))
        q = s["q"][:, t0:t1].float().view(b, t1 - t0, G, H // G, P).permute(0, 2, 3, 1, 4)
        k = torch.cat([s["k"][:, x] for x in parts], 1).float().permute(0, 2, 3, 1)[:, :, None]
        x = (s["scale"] * (q @ k)).masked_fill(~seen, -math.inf)
        m = x.amax(-1, keepdim=True)
        e = (x - m).exp()
        total = e.sum(-1, keepdim=True)
        each(t0, t1, parts, q, e / total, m + total.log())


def _rows(x):  # [b, G, R, queries, P] -> [b, queries, H, P]
    b, G, R, n, P = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(b, n, G * R, P)


def _plain_forward(s, kept=None):
    b, L, H, P = s["q"].shape
    on = _present(s, b, L)
    v = s["v"].float() * on[:, :, None, None]
    o, lse = torch.empty(b, L, H, P, device=DEV), torch.empty(b, H, L, device=DEV)

    def each(t0, t1, parts, q, p, logs):
        vb = torch.cat([v[:, x] for x in parts], 1).permute(0, 2, 1, 3)[:, :, None]
        o[:, t0:t1] = _rows(p @ vb)
        lse[:, :, t0:t1] = logs.view(b, H, t1 - t0)

    _plain_blocks(s, each)
    return o * on[:, :, None, None], lse * on[:, None, :]


def _plain_prefill(s):
    o, _ = _plain_forward(s)
    L, entries = s["q"].shape[1], s["k_cache"].shape[1]
    W, n = s["window"], s["sinks"]
    j = torch.arange(entries, device=DEV)[None, :]
    V = (s["valid_len"].clamp(0, L) if s["valid_len"] is not None else torch.full((s["q"].shape[0],), L, device=DEV))[:, None]
    # the newest present token of every entry: the entry's own residue, up to V - 1
    t = torch.where(j < n, j, j + torch.div(V - 1 - j, W, rounding_mode="floor").clamp(min=0) * W)
    row, at = (t < V).nonzero(as_tuple=True)
    slot, token = s["index"].long()[row], t[row, at]
    s["k_cache"][slot, at] = s["k"][row, token]
    s["v_cache"][slot, at] = s["v"][row, token]
    return dict(o=o.to(s["q"].dtype), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_train(s):
    b, L, H, P = s["q"].shape
    on = _present(s, b, L)
    v, do = s["v"].float() * on[:, :, None, None], s["do"].float() * on[:, :, None, None]
    kf = s["k"].float()
    G = s["k"].shape[2]
    o, lse, dq = torch.empty(b, L, H, P, device=DEV), torch.empty(b, H, L, device=DEV), torch.empty(b, L, H, P, device=DEV)
    dk, dv = torch.zeros(b, L, G, P, device=DEV), torch.zeros(b, L, G, P, device=DEV)

    def each(t0, t1, parts, q, p, logs):
        vb = torch.cat([v[:, x] for x in parts], 1).permute(0, 2, 1, 3)[:, :, None]
        kb = torch.cat([kf[:, x] for x in parts], 1).permute(0, 2, 1, 3)[:, :, None]
        out = p @ vb
        o[:, t0:t1] = _rows(out)
        lse[:, :, t0:t1] = logs.view(b, H, t1 - t0)
        g = do[:, t0:t1].view(b, t1 - t0, G, H // G, P).permute(0, 2, 3, 1, 4)
        ds = s["scale"] * p * (g @ vb.transpose(-1, -2) - (g * out).sum(-1, keepdim=True))
        dq[:, t0:t1] = _rows(ds @ kb)
        dkb, dvb = (ds.transpose(-1, -2) @ q).sum(2), (p.transpose(-1, -2) @ g).sum(2)
        at = 0
        for x in parts:
            n = x.stop - x.start
            dk[:, x] += dkb[:, :, at:at + n].permute(0, 2, 1, 3)
            dv[:, x] += dvb[:, :, at:at + n].permute(0, 2, 1, 3)
            at += n

    _plain_blocks(s, each)
    T, live = s["q"].dtype, on[:, :, None, None]
    return dict(o=(o * live).to(T), lse=lse * on[:, None, :], dq=(dq * live).to(T), dk=(dk * live).to(T), dv=(dv * live).to(T))


def _plain_step(s):
    b, H, P = s["q"].shape
    G, entries = s["k"].shape[1], s["k_cache"].shape[1]
    pos, slot, n = s["position"].long(), s["index"].long(), s["sinks"]
    at = torch.where(pos < n, pos, n + (pos - n) % s["window"])
    s["k_cache"][slot, at], s["v_cache"][slot, at] = s["k"], s["v"]
    k, v = s["k_cache"][slot].float(), s["v_cache"][slot].float()
    seen = torch.arange(entries, device=DEV)[None, :] < (pos + 1)[:, None]
    x = s["scale"] * (s["q"].float().view(b, G, H // G, P) @ k.permute(0, 2, 3, 1))
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    e = (x - x.amax(-1, keepdim=True)).exp()
    o = (e / e.sum(-1, keepdim=True)) @ (v * seen[:, :, None, None]).permute(0, 2, 1, 3)
    return dict(o=o.view(b, H, P).to(s["q"].dtype), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _act(s, x):  # the activation and its derivative
    g = torch.sigmoid(x)
    return (x * g, g * (1 + x * (1 - g))) if s["act"] == "silu" else (g, g * (1 - g))


def _plain_exit(s, train=False):
    R, D = s["x"].shape
    x, w = s["x"].float(), s["weight"]
    b = s["bias"] if s["bias"] is not None else torch.zeros_like(w)
    z = s["gate"].float() if s["gate"] is not None else None
    a, da = _act(s, z) if z is not None else (None, None)
    u = (x * a if s["first"] else x).view(R, s["groups"], -1)
    if s["center"]:
        u = u - u.mean(-1, keepdim=True)
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + s["eps"])
    n = (u * rstd).view(R, D)
    y = n * w + b
    if z is None:
        out, slope = _act(s, y)
    else:
        out = y if s["first"] else y * a
    if not train:
        return dict(y=out.to(s["x"].dtype))
    dy = s["dy"].float()
    dn = dy * slope if z is None else (dy if s["first"] else dy * a)
    dw, db = (dn * n).sum(0), dn.sum(0)
    t, nv = (dn * w).view(u.shape), n.view(u.shape)
    du = t - nv * (t * nv).mean(-1, keepdim=True)
    if s["center"]:
        du = du - t.mean(-1, keepdim=True)
    du = (rstd * du).view(R, D)
    dx = du * a if s["first"] else du
    dz = None if z is None else (du * x * da if s["first"] else dy * y * da)
    T = s["x"].dtype
    return dict(y=out.to(T), dx=dx.to(T), dgate=None if dz is None else dz.to(T), dweight=dw,
                dbias=db if s["bias"] is not None else None)


def _plain_scan_step(s):
    H, G = s["x"].shape[1], s["B"].shape[1]
    heads = torch.arange(H, device=DEV) // (H // G)
    x, at = s["x"].float(), s["index"].long()
    B, C = s["B"].float()[:, heads], s["C"].float()[:, heads]
    S = s["state"][at] * (s["dt"] * s["A"]).exp()[..., None, None]
    S = S + (s["dt"][..., None] * x)[..., None] * B[:, :, None, :]
    s["state"][at] = S
    y = (S * C[:, :, None, :]).sum(-1) + s["D"][:, None] * x
    return dict(y=y.to(s["x"].dtype), state=s["state"])


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["op"]
    if not own:
        return {"prefill": _plain_prefill, "train": _plain_train, "step": _plain_step, "exit": _plain_exit,
                "exit_train": lambda s: _plain_exit(s, True), "scan_step": _plain_scan_step}[op](s)
    from state_space_model_mamba_gb300 import norm, ssd, window
    if op == "prefill":
        o, _ = window.window_forward(s["q"], s["k"], s["v"], s["window"], s["sinks"], scale=s["scale"], valid_len=s["valid_len"],
                                     return_lse=False)
        window.window_fill(s["k"], s["v"], s["k_cache"], s["v_cache"], s["window"], s["sinks"], valid_len=s["valid_len"],
                           cache_index=s["index"])
        return dict(o=o, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "train":
        o, lse = window.window_forward(s["q"], s["k"], s["v"], s["window"], s["sinks"], scale=s["scale"], valid_len=s["valid_len"])
        grads = window.window_backward(s["q"], s["k"], s["v"], o, lse, s["do"], s["window"], s["sinks"], scale=s["scale"],
                                       valid_len=s["valid_len"])
        return dict(o=o, lse=lse, **grads)
    if op == "step":
        o = window.window_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["position"], s["window"], s["sinks"],
                               scale=s["scale"], cache_index=s["index"])
        return dict(o=o, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "scan_step":
        y = ssd.ssd_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["state"], state_index=s["index"])
        return dict(y=y, state=s["state"])
    form = dict(groups=s["groups"], eps=s["eps"], center=s["center"], activation=s["act"], gate_first=s["first"])
    y = norm.group_norm_gated(s["x"], s["weight"], bias=s["bias"], gate=s["gate"], **form)
    if op == "exit":
        return dict(y=y)
    return dict(y=y, **norm.group_norm_gated_backward(s["dy"], s["x"], s["weight"], bias=s["bias"], gate=s["gate"], **form))


def _pairs(L, W, sinks):
    """Visible pairs of a sequence of L tokens: min(t + 1, W) in the window, and sinks in front of it."""
    n = min(L, W)
    total = n * (n + 1) // 2 + (L - n) * W
    m = max(0, L - W)  # tokens with something in front of their window
    k = min(sinks, m)
    return total + k * (k + 1) // 2 + (m - k) * k


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("exit", "exit_train"):
        R, D, gate = case["rows"], case["D"], case["gate"] != "none"
        small = 4 * D * (1 + case["bias"])
        if op == "exit":
            return dict(bytes=R * D * e * (2 + gate) + small, flops=12 * R * D)
        return dict(bytes=R * D * e * (4 + 2 * gate) + 2 * small, flops=36 * R * D)
    b, H, G, P = case["b"], case["H"], case["G"], case["P"]
    if op == "scan_step":
        N = case["N"]
        return dict(bytes=b * (8 * H * P * N + e * (2 * G * N + 2 * H * P) + 4 * H + 4) + 8 * H, flops=5 * b * H * P * N)
    entries = case["sinks"] + case["window"]
    if op == "step":
        n = 0.75 * entries if case["young"] else entries  # entries of a request, on average
        return dict(bytes=int(b * (2 * n * G * P * e + 2 * H * P * e + 4 * G * P * e + 8)), flops=int(4 * b * H * P * n))
    L = case["L"]
    share = 0.625 if case["ragged"] and L >= 8 else 1.0  # lengths are spread evenly over L / 4 .. L
    pairs, t = b * H * share * _pairs(L, case["window"], case["sinks"]), b * L * share
    if op == "prefill":
        kept = b * min(entries, L)
        return dict(bytes=int(t * P * e * (2 * H + 2 * G) + kept * 2 * G * P * e), flops=int(4 * P * pairs))
    return dict(bytes=int(t * P * e * (4 * H + 4 * G) + 4 * t * H), flops=int(14 * P * pairs))


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_attn(s, train):
    """Head by head: blocks of 256 queries against every key from the window's first on, and the sinks."""
    b, L, H, P = s["q"].shape
    G, W, sinks, c = s["k"].shape[2], s["window"], s["sinks"], s["scale"]
    f8 = torch.float64
    out = dict(o=torch.zeros(b, L, H, P, dtype=f8, device=DEV))
    if train:
        out.update(lse=torch.zeros(b, H, L, dtype=f8, device=DEV), dq=torch.zeros(b, L, H, P, dtype=f8, device=DEV),
                   dk=torch.zeros(b, L, G, P, dtype=f8, device=DEV), dv=torch.zeros(b, L, G, P, dtype=f8, device=DEV))
    lengths = [L] * b if s["valid_len"] is None else [min(L, max(0, x)) for x in s["valid_len"].tolist()]
    for i, V in enumerate(lengths):
        for first in range(0, V, 256):
            last = min(V, first + 256)
            start = max(0, first - W + 1)
            head = min(sinks, start)
            seen = torch.cat([torch.arange(head, device=DEV), torch.arange(start, last, device=DEV)])
            at = torch.arange(first, last, device=DEV)
            gap = at[:, None] - seen[None, :]
            hidden = (gap < 0) | ((gap >= W) & (seen[None, :] >= sinks))
            K, Vv = s["k"][i][seen].double().transpose(0, 1), s["v"][i][seen].double().transpose(0, 1)  # [G, keys, P]
            Q = s["q"][i, first:last].double().transpose(0, 1).reshape(G, -1, P)                          # [G, R queries, P]
            x = torch.bmm(Q, K.transpose(1, 2)).mul_(c).view(G, H // G, last - first, -1)
            x.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[..., None]).view(G, Q.shape[1], -1)
            O = torch.bmm(p, Vv)
            out["o"][i, first:last] = O.view(H, last - first, P).transpose(0, 1)
            if not train:
                continue
            out["lse"][i, :, first:last] = lse.reshape(H, -1)
            dO = s["do"][i, first:last].double().transpose(0, 1).reshape(G, -1, P)
            dp = torch.bmm(dO, Vv.transpose(1, 2))
            dx = c * p * (dp - (p * dp).sum(-1, keepdim=True))
            out["dq"][i, first:last] = torch.bmm(dx, K).view(H, last - first, P).transpose(0, 1)
            out["dk"][i].index_add_(0, seen, torch.bmm(dx.transpose(1, 2), Q).transpose(0, 1))
            out["dv"][i].index_add_(0, seen, torch.bmm(p.transpose(1, 2), dO).transpose(0, 1))
    return out


def _exact_prefill(s):
    out = _exact_attn(s, False)
    L, W, n = s["q"].shape[1], s["window"], s["sinks"]
    for name, x in (("k_cache", s["k"]), ("v_cache", s["v"])):
        cache = s[name].double()
        for i in range(x.shape[0]):
            V = L if s["valid_len"] is None else min(L, max(0, int(s["valid_len"][i])))
            slot = int(s["index"][i])
            cache[slot, :min(n, V)] = x[i, :min(n, V)].double()
            t = torch.arange(max(n, V - W), max(n, V), device=DEV)
            cache[slot, n + (t - n) % W] = x[i, t].double()
        out[name] = cache
    return out


def _exact_step(s):
    b, H, P = s["q"].shape
    G, W, n = s["k"].shape[1], s["window"], s["sinks"]
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    o = torch.empty(b, H, P, dtype=torch.float64, device=DEV)
    for i in range(b):
        t, slot = int(s["position"][i]), int(s["index"][i])
        at = t if t < n else n + (t - n) % W
        kc[slot, at], vc[slot, at] = s["k"][i], s["v"][i]
        m = min(t + 1, n + W)
        K, V = kc[slot, :m].double().transpose(0, 1), vc[slot, :m].double().transpose(0, 1)
        p = torch.softmax(s["scale"] * torch.bmm(s["q"][i].double().view(G, H // G, P), K.transpose(1, 2)), -1)
        o[i] = torch.bmm(p, V).view(H, P)
    return dict(o=o, k_cache=kc.double(), v_cache=vc.double())


def _exact_exit(s, train):
    leaves = {k: s[k].double().requires_grad_(train) for k in ("x", "gate", "weight", "bias") if s[k] is not None}
    R, D = s["x"].shape

    def act(t):
        return t / (1 + torch.exp(-t)) if s["act"] == "silu" else 1 / (1 + torch.exp(-t))

    with torch.set_grad_enabled(train):
        u = leaves["x"] * act(leaves["gate"]) if s["first"] else leaves["x"]
        u = u.reshape(R, s["groups"], D // s["groups"])
        mu = u.mean(-1, keepdim=True) if s["center"] else 0.0
        n = (u - mu) / torch.sqrt(((u - mu) ** 2).mean(-1, keepdim=True) + s["eps"])
        y = n.reshape(R, D) * leaves["weight"]
        if "bias" in leaves:
            y = y + leaves["bias"]
        if "gate" not in leaves:
            y = act(y)
        elif not s["first"]:
            y = y * act(leaves["gate"])
    if not train:
        return dict(y=y)
    names = list(leaves)
    grads = dict(zip(names, torch.autograd.grad(y, [leaves[k] for k in names], s["dy"].double())))
    return dict(y=y.detach(), dx=grads["x"], dgate=grads.get("gate"), dweight=grads["weight"], dbias=grads.get("bias"))


def _exact_scan_step(s):
    rep = s["x"].shape[1] // s["B"].shape[1]
    B, C = (s[k].double().repeat_interleave(rep, dim=1) for k in ("B", "C"))
    x, dt, state, at = s["x"].double(), s["dt"].double(), s["state"].double(), s["index"].long()
    S = state[at] * torch.exp(dt * s["A"].double())[..., None, None] + torch.einsum("bh,bhp,bhn->bhpn", dt, x, B)
    state[at] = S
    return dict(y=torch.einsum("bhpn,bhn->bhp", S, C) + s["D"].double()[:, None] * x, state=state)


def exact(case, seed):
    op = case["op"]
    if op in ("prefill", "train"):
        # fp64 products at some 0.8 TFLOP/s, a few passes over the pairs, launches
        pairs = case["b"] * case["H"] * case["L"] * min(case["L"], case["window"] + 256 + case["sinks"])
        if pairs * (case["P"] * (4 if op == "prefill" else 14) / 8e11 + 4e-11) + case["b"] * case["L"] / 256 * 1e-3 > 18.0:
            return None
    s = prepare(case, seed)
    if op in ("prefill", "train"):
        return _exact_prefill(s) if op == "prefill" else _exact_attn(s, True)
    if op in ("exit", "exit_train"):
        return _exact_exit(s, op == "exit_train")
    return _exact_step(s) if op == "step" else _exact_scan_step(s)
