"""The operators measured here: the gated delta rule (forward, backward, one-token
step) and the residual addition with a root-mean-square norm (outputs in the
stream's type or in 8 bits with scales, and its backward).

``run`` computes them either in a plain form (elementary torch operations in
fp32, rounded once at the end) or, with ``own`` set, through this package.
``exact`` is the same in 64 bits, token by token, from the definitions:

  delta rule, per batch and head (key group g = h / (H / G)), state S [P, N]:
      S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) (x) k_t,  a_t = exp(g_t)
      o_t = scale S_t q_t            (tokens at or past valid_len are absent)
  norm, per row:  h = x + residual (kept in the stream's type),
      y = h / sqrt(mean(h^2) + eps) * weight;  8 bits: y / s in e4m3 with
      s = max |y| / 448 over the row or over each group of columns.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens per chunk of the plain form


# ------------------------------------------------------------------ the cases
def _delta(name, op, b, L, H, P, N, G, dtype="bf16", dt_mu=-4.0, init=False, ragged=False):
    return dict(name=name, op=op, b=b, L=L, H=H, P=P, N=N, G=G, dtype=dtype, dt_mu=dt_mu, init=init, ragged=ragged)


def listed():
    return [
        # a short prompt of one request, continuing from a cached state: latency counts
        _delta("fwd_prompt", "delta_fwd", 1, 333, 16, 128, 128, 8, init=True),
        # a prefill batch of padded prompts of different lengths (the grouped, padded workload's shape)
        _delta("fwd_grouped_padded", "delta_fwd", 8, 4096, 64, 64, 128, 8, dt_mu=-2.0, init=True, ragged=True),
        # one document of 131072 tokens, 32 heads with a key head each (the long-sequence workload's shape)
        _delta("fwd_long", "delta_fwd", 1, 131072, 32, 64, 128, 32, dt_mu=-3.0),
        # fp32 debugging and gradient-check runs at small sizes: forward and backward
        _delta("fwd_f32", "delta_fwd", 2, 515, 4, 32, 48, 2, dtype="f32", init=True),
        _delta("bwd_f32", "delta_bwd", 2, 129, 4, 32, 48, 2, dtype="f32", init=True),
        # training step of the 130M layer: heads of 64, every head with its own keys
        _delta("bwd_130m", "delta_bwd", 4, 2048, 24, 64, 128, 24),
        # training step of the 2.7B layer, keys shared by five heads
        _delta("bwd_2p7b", "delta_bwd", 2, 8192, 80, 64, 128, 16, dt_mu=-2.0),
        # one decoded token of one request, and of a batch drawn from a larger pool of states
        dict(name="step_one", op="step", b=1, H=80, P=64, N=128, G=16, slots=4, dtype="bf16"),
        dict(name="step_batch", op="step", b=192, H=80, P=64, N=128, G=16, slots=256, dtype="bf16"),
        # the block's entry norm: a decode batch in bf16, and the 2.7B layer's tokens into 8 bits
        dict(name="norm_decode", op="norm", rows=24, D=2560, dtype="bf16", out="same", group=0),
        dict(name="norm_fp8", op="norm", rows=16384, D=2560, dtype="bf16", out="fp8", group=128),
        # its training backward at the same size
        dict(name="norm_bwd", op="norm_bwd", rows=16384, D=2560, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "step", "norm", "norm_bwd"])
    if op in ("delta_fwd", "delta_bwd"):
        # mostly bf16 at the head sizes of real layers; fp32 at small ones
        if rng.random() < 0.8:
            P, N, dtype = rng.choice([64, 64, 128, 96]), rng.choice([128, 128, 64, 80]), "bf16"
            most, H = (3e10 if op == "delta_fwd" else 1e10), 4 * _log(rng, 1, 20)
        else:
            P, N, dtype = 4 * rng.randint(2, 12), 4 * rng.randint(2, 16), "f32"
            most, H = 1.5e7, 4
        G = H // rng.choice([1, 2, 4])
        b = rng.choice([1, 1, 2, 3, 4])
        # the work of all tokens and heads stays below the largest listed case's
        L = _log(rng, 1, min(8192 if op == "delta_bwd" else 65536, int(most / (b * H * P * N))))
        return dict(op=op, b=b, L=L, H=H, P=P, N=N, G=G, dtype=dtype, dt_mu=rng.choice([-4.0, -3.0, -2.0]),
                    init=rng.random() < 0.5, ragged=rng.random() < 0.4)
    if op == "step":
        H, b = 4 * _log(rng, 1, 20), _log(rng, 1, 192)
        return dict(op=op, b=b, H=H, P=rng.choice([64, 64, 128, 40]), N=rng.choice([128, 128, 64, 72]),
                    G=H // rng.choice([1, 2, 4]), slots=b + rng.randint(0, 64), dtype=rng.choice(["bf16", "bf16", "f32"]))
    D = rng.choice([128 * rng.randint(2, 40), rng.randint(200, 5200), 2560])
    rows = _log(rng, 1, 40_000_000 // D)
    if op == "norm":
        out = rng.choice(["same", "fp8", "fp8"])
        group = 128 if out == "fp8" and D % 128 == 0 and rng.random() < 0.5 else 0
        return dict(op=op, rows=rows, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]), out=out, group=group)
    return dict(op=op, rows=rows, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    gen, T, op = _gen(seed), TYPES[case["dtype"]], case["op"]

    def randn(*s):
        return torch.randn(*s, generator=gen, device=DEV)

    s = dict(op=op)
    if op in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        s["x"] = randn(R, D).to(T)
        s["weight"] = 1.0 + 0.1 * randn(D)
        s["eps"] = 1e-5
        if op == "norm":
            s["residual"] = (3.0 * randn(R, D)).to(T)
            s["out"], s["group"] = case["out"], case["group"]
        else:
            s["x"] = (3.0 * randn(R, D)).to(T)      # the stored stream
            s["dy"], s["d_stream"] = randn(R, D).to(T), randn(R, D).to(T)
        return s
    b, H, P, N, G = case["b"], case["H"], case["P"], case["N"], case["G"]
    lead = (b,) if op == "step" else (b, case["L"])

    def unit(x):  # keys and queries come out of a SiLU and an L2 norm
        x = x * torch.sigmoid(x)
        return (x / x.norm(dim=-1, keepdim=True)).to(T)

    s["q"], s["k"] = unit(randn(*lead, G, N)), unit(randn(*lead, G, N))
    s["v"] = randn(*lead, H, P).to(T)
    rate = torch.exp(math.log(16.0) * torch.rand(H, generator=gen, device=DEV))
    gl = (b, H) if op == "step" else (b, H, case["L"])
    dt = torch.nn.functional.softplus(randn(*gl) + case.get("dt_mu", -4.0))
    s["g"] = -rate.view(1, H, *([1] * (len(gl) - 2))) * dt
    s["beta"] = torch.sigmoid(randn(*gl))
    s["scale"] = N ** -0.5
    if op == "step":
        s["state"] = 0.3 * randn(case["slots"], H, P, N)
        s["index"] = torch.randperm(case["slots"], generator=gen, device=DEV)[:b].to(torch.int32)
        return s
    s["init"] = 0.1 * randn(b, H, P, N) if case["init"] else None
    s["valid_len"] = None
    if case["ragged"]:
        L = case["L"]
        s["valid_len"] = torch.randint(min(L, max(1, L // 4)), L + 1, (b,), generator=gen, device=DEV).to(torch.int32)
    if op == "delta_bwd":
        s["do"] = randn(b, case["L"], H, P).to(T)
        s["d_final"] = randn(b, H, P, N)
    return s


# ------------------------------------------------------------------ plain forms
def _chunked(s):
    """fp32 copies per (b, H, chunk): q, k, v, gamma, beta and the decay matrix."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    b, L, G, N = q.shape
    H, P = v.shape[2:]
    n = -(-L // CHUNK)
    live = torch.arange(n * CHUNK, device=q.device)[None, :] < (
        s["valid_len"].clamp(0, L)[:, None] if s["valid_len"] is not None else torch.full((b, 1), L, device=q.device))

    def tokens(x):  # [b, L, h, X] -> [b, h, n, CHUNK, X], absent tokens zero
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * CHUNK - L)) * live[:, :, None, None]
        return x.view(b, n, CHUNK, x.shape[2], x.shape[3]).permute(0, 3, 1, 2, 4)

    def gates(x):
        x = torch.nn.functional.pad(x.float(), (0, n * CHUNK - L)) * live[:, None, :]
        return x.view(b, H, n, CHUNK)

    heads = torch.arange(H, device=q.device) // (H // G)
    qc, kc, vc = tokens(q)[:, heads], tokens(k)[:, heads], tokens(v)
    gam, beta = gates(s["g"]).cumsum(-1), gates(s["beta"])
    diff = gam[..., :, None] - gam[..., None, :]
    i = torch.arange(CHUNK, device=q.device)
    low = i[:, None] >= i[None, :]
    decay = torch.where(low, diff, torch.full_like(diff, -math.inf)).exp()
    return qc, kc, vc, gam, beta, decay, live, heads


def _inverse(Lm):
    """(I + Lm)^-1 of strictly lower triangular matrices, row by row."""
    T = torch.eye(CHUNK, device=Lm.device).expand(Lm.shape).clone()
    for r in range(1, CHUNK):
        T[..., r, :r] = -(Lm[..., r:r + 1, :r] @ T[..., :r, :r]).squeeze(-2)
    return T


def _plain_states(s, c):
    """T, the errors Z = v - read, the state before every chunk and the last one."""
    qc, kc, vc, gam, beta, decay = c[:6]
    b, H, n = gam.shape[:3]
    kk = kc @ kc.transpose(-1, -2)
    T = _inverse(torch.tril(decay * kk, -1) * beta[..., None, :])
    eg = gam.exp()[..., None]
    Z0, W = T @ vc, T @ (eg * kc)
    tail = (gam[..., -1:] - gam).exp()[..., None]
    kt = (tail * kc).transpose(-1, -2)
    end = gam[..., -1].exp()[..., None, None]
    S = torch.zeros(b, H, kc.shape[-1], vc.shape[-1], device=vc.device)
    if s["init"] is not None:
        S = s["init"].transpose(-1, -2).float()
    states, Zs = [], []
    for j in range(n):
        states.append(S)
        Z = Z0[:, :, j] - W[:, :, j] @ S
        Zs.append(Z)
        S = end[:, :, j] * S + kt[:, :, j] @ (beta[:, :, j, :, None] * Z)
    return kk, T, torch.stack(Zs, 2), torch.stack(states, 2), S, eg, tail, end


def _untokens(x, L):
    b, h, n, C, X = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(b, n * C, h, X)[:, :L]


def _plain_delta_fwd(s):
    c = _chunked(s)
    qc, kc, vc, gam, beta, decay, live, _ = c
    _, _, Z, S0, S, eg, _, _ = _plain_states(s, c)
    A = decay * (qc @ kc.transpose(-1, -2))
    o = s["scale"] * (eg * (qc @ S0) + A @ (beta[..., None] * Z))
    o = _untokens(o, s["v"].shape[1]) * live[:, :s["v"].shape[1], None, None]
    return dict(o=o.to(s["v"].dtype), final_state=S.transpose(-1, -2).contiguous())


def _plain_delta_bwd(s):
    c = _chunked(s)
    qc, kc, vc, gam, beta, decay, live, heads = c
    kk, T, Z, S0, S, eg, tail, end = _plain_states(s, c)
    b, L, G, N = s["q"].shape
    H, P = s["v"].shape[2:]
    n = gam.shape[2]
    do = torch.nn.functional.pad(s["do"].float(), (0, 0, 0, 0, 0, n * CHUNK - L)) * live[:, :, None, None]
    do = s["scale"] * do.view(b, n, CHUNK, H, P).permute(0, 3, 1, 2, 4)
    A = decay * (qc @ kc.transpose(-1, -2))
    bt = beta[..., None]
    U = bt * Z
    kt = tail * kc
    dU_own, dS_own = A.transpose(-1, -2) @ do, qc.transpose(-1, -2) @ (eg * do)
    dS = s["d_final"].transpose(-1, -2).float()
    Tt, ek = T.transpose(-1, -2), (eg * kc).transpose(-1, -2)
    dUs, Ys, dSs = [None] * n, [None] * n, [None] * n
    for j in reversed(range(n)):
        dSs[j] = dS
        dUs[j] = dU_own[:, :, j] + kt[:, :, j] @ dS
        Ys[j] = Tt[:, :, j] @ (bt[:, :, j] * dUs[j])
        dS = end[:, :, j] * dS + dS_own[:, :, j] - ek[:, :, j] @ Ys[j]
    dU, Y, dSe = torch.stack(dUs, 2), torch.stack(Ys, 2), torch.stack(dSs, 2)
    R = torch.tril(Y @ Z.transpose(-1, -2), -1) * decay
    M = -R * beta[..., None, :]
    Nm = decay * (do @ U.transpose(-1, -2))
    S0t = S0.transpose(-1, -2)
    dq = eg * (do @ S0t) + Nm @ kc
    dk_row = M @ kc - eg * (Y @ S0t)
    write = tail * (U @ dSe.transpose(-1, -2))
    dk_col = Nm.transpose(-1, -2) @ qc + M.transpose(-1, -2) @ kc + write
    dbeta = (Z * dU).sum(-1) - (R * kk).sum(-2)
    dgam = (qc * dq).sum(-1) + (kc * (dk_row - dk_col)).sum(-1)
    last = end[..., 0, 0] * (S0 * dSe).sum((-1, -2)) + (kc * write).sum((-1, -2))
    dg = dgam.flip(-1).cumsum(-1).flip(-1) + last[..., None]
    per = H // G

    def group(x):
        return _untokens(x.view(b, G, per, *x.shape[2:]).sum(2), L).to(s["q"].dtype)

    def gate(x):
        return (x.reshape(b, H, n * CHUNK) * live[:, None, :])[..., :L].contiguous()

    return dict(dq=group(dq), dk=group(dk_row + dk_col), dv=_untokens(Y, L).to(s["v"].dtype), dg=gate(dg),
                dbeta=gate(dbeta), d_init=dS.transpose(-1, -2).contiguous() if s["init"] is not None else None)


def _plain_step(s):
    H, G = s["v"].shape[1], s["q"].shape[1]
    heads = torch.arange(H, device=s["v"].device) // (H // G)
    q, k, v = s["q"].float()[:, heads], s["k"].float()[:, heads], s["v"].float()
    at = s["index"].long()
    S = s["state"][at] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (v - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., None] * k[:, :, None, :]
    s["state"][at] = S
    o = s["scale"] * (S * q[:, :, None, :]).sum(-1)
    return dict(o=o.to(s["v"].dtype), state=s["state"])


E4M3_MAX = 448.0


def _plain_norm(s):
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    if s["out"] == "same":
        return dict(y=y.to(h.dtype), stream=h)
    R, D = y.shape
    parts = y.view(R, -1, s["group"] or D)
    scale = parts.abs().amax(-1) / E4M3_MAX
    y8 = (parts / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(y8=y8.view(R, D), scale=scale, stream=h)


def _plain_norm_bwd(s):
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"])
    t = dy * s["weight"]
    dx = s["d_stream"].float() + r * (t - h * (r * r * (t * h).mean(-1, keepdim=True)))
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * h * r).sum(0))


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["op"]
    if not own:
        return {"delta_fwd": _plain_delta_fwd, "delta_bwd": _plain_delta_bwd, "step": _plain_step,
                "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[op](s)
    from state_space_model_mamba_gb300 import delta, norm
    if op == "delta_fwd":
        o, fin = delta.delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], init_state=s["init"],
                                     valid_len=s["valid_len"])
        return dict(o=o, final_state=fin)
    if op == "delta_bwd":
        return delta.delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], scale=s["scale"],
                                    init_state=s["init"], d_final_state=s["d_final"], valid_len=s["valid_len"],
                                    want_d_init=s["init"] is not None)
    if op == "step":
        o = delta.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"],
                             state_index=s["index"])
        return dict(o=o, state=s["state"])
    if op == "norm":
        if s["out"] == "same":
            y, stream = norm.add_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"])
            return dict(y=y, stream=stream)
        y8, scale, stream = norm.add_rms_norm_fp8(s["x"], s["weight"], s["eps"], residual=s["residual"],
                                                  group=s["group"])
        return dict(y8=y8, scale=scale, stream=stream)
    dx, dw = norm.add_rms_norm_backward(s["dy"], s["x"], s["weight"], s["eps"], d_stream=s["d_stream"])
    return dict(dx=dx, dweight=dw)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        if op == "norm_bwd":
            return dict(bytes=4 * R * D * e + 8 * D, flops=12 * R * D)
        if case["out"] == "same":
            return dict(bytes=4 * R * D * e + 4 * D, flops=6 * R * D)
        return dict(bytes=3 * R * D * e + R * D + 4 * R * (D // (case["group"] or D)) + 4 * D, flops=8 * R * D)
    b, H, P, N, G = case["b"], case["H"], case["P"], case["N"], case["G"]
    if op == "step":
        return dict(bytes=b * (8 * H * P * N + e * (2 * G * N + 2 * H * P) + 8 * H + 4), flops=7 * b * H * P * N)
    t, C = b * case["L"], min(CHUNK, case["L"])
    state = 4 * b * H * P * N
    qk, vo = t * 2 * G * N * e, t * H * P * e
    if op == "delta_fwd":
        # per token and head: k S, q S and the update (6 P N); the chunk's causal halves of k k, q k, T v, A u
        return dict(bytes=qk + 2 * vo + 8 * t * H + state * (1 + case["init"]),
                    flops=t * H * (6 * P * N + 2 * C * N + 2 * C * P))
    # the forward's states again, then per token and head k dS, q do, k y, do S, y S, u dS (12 P N) and the
    # causal halves of k k, q k, T, A do, do u, y z and four products with q or k
    return dict(bytes=2 * qk + 3 * vo + 16 * t * H + state * (1 + 2 * case["init"]),
                flops=t * H * (4 * P * N + 12 * P * N + 6 * C * N + 5 * C * P))


# ------------------------------------------------------------------ 64 bits, from the definitions
def _token_form(s):
    H, G = s["v"].shape[2], s["q"].shape[2]
    rep = H // G

    def tok(x, r=1):  # token first: [L, b, H, X]
        return x.double().permute(1, 0, 2, 3).repeat_interleave(r, dim=2)

    q, k, v = tok(s["q"], rep), tok(s["k"], rep), tok(s["v"])
    g, beta = s["g"].double().permute(2, 0, 1), s["beta"].double().permute(2, 0, 1)
    L, b = v.shape[:2]
    vl = s["valid_len"].long() if s["valid_len"] is not None else torch.full((b,), L, device=v.device)
    on = (torch.arange(L, device=v.device)[:, None] < vl[None, :]).double()[:, :, None]
    a, beta = torch.exp(g * on)[..., None, None], (beta * on)[..., None]
    S = torch.zeros(b, H, v.shape[-1], k.shape[-1], dtype=torch.float64, device=v.device)
    if s["init"] is not None:
        S = s["init"].double().clone()
    return q, k, v, a, beta, on, S


def _exact_delta_fwd(s):
    q, k, v, a, beta, on, S = _token_form(s)
    o = torch.empty_like(v)
    for t in range(v.shape[0]):
        S = S * a[t]
        u = beta[t] * (v[t] - (S @ k[t].unsqueeze(-1)).squeeze(-1))
        S = torch.baddbmm(S.flatten(0, 1), u.flatten(0, 1).unsqueeze(-1), k[t].flatten(0, 1).unsqueeze(1)).view_as(S)
        o[t] = (S @ q[t].unsqueeze(-1)).squeeze(-1)
    o = s["scale"] * o * on[..., None]
    return dict(o=o.permute(1, 0, 2, 3).contiguous(), final_state=S)


def _exact_delta_bwd(s):
    q, k, v, a, beta, on, S = _token_form(s)
    L, b, H, P = v.shape
    G = s["q"].shape[2]
    seg = 64
    do = s["scale"] * s["do"].double().permute(1, 0, 2, 3) * on[..., None]
    kept = []
    for t in range(L):  # forward, the state kept before every segment
        if t % seg == 0:
            kept.append(S)
        S = S * a[t]
        S = S + (beta[t] * (v[t] - (S @ k[t].unsqueeze(-1)).squeeze(-1))).unsqueeze(-1) * k[t].unsqueeze(-2)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = (torch.empty(L, b, H, dtype=torch.float64, device=v.device) for _ in range(2))
    dS = s["d_final"].double()
    for first in reversed(range(0, L, seg)):
        S, last = kept.pop(), min(L, first + seg)
        before, after, err = [], [], []
        for t in range(first, last):
            S = S * a[t]
            before.append(S)  # after the decay
            z = v[t] - (S @ k[t].unsqueeze(-1)).squeeze(-1)
            err.append(z)
            S = S + (beta[t] * z).unsqueeze(-1) * k[t].unsqueeze(-2)
            after.append(S)
        for t in reversed(range(first, last)):
            Sd, z, Sa = before.pop(), err.pop(), after.pop()
            dq[t] = (do[t].unsqueeze(-2) @ Sa).squeeze(-2)
            dS = dS + do[t].unsqueeze(-1) * q[t].unsqueeze(-2)
            dSk = (dS @ k[t].unsqueeze(-1)).squeeze(-1)
            dbeta[t] = (dSk * z).sum(-1)
            dz = beta[t] * dSk
            dv[t] = dz
            dk[t] = ((beta[t] * z).unsqueeze(-2) @ dS - dz.unsqueeze(-2) @ Sd).squeeze(-2)
            dS = dS - dz.unsqueeze(-1) * k[t].unsqueeze(-2)
            dg[t] = (dS * Sd).sum((-1, -2))
            dS = dS * a[t]

    def group(x):
        return (x * on[..., None]).view(L, b, G, H // G, -1).sum(3).permute(1, 0, 2, 3).contiguous()

    return dict(dq=group(dq), dk=group(dk), dv=(dv * on[..., None]).permute(1, 0, 2, 3).contiguous(),
                dg=(dg * on).permute(1, 2, 0).contiguous(), dbeta=(dbeta * on).permute(1, 2, 0).contiguous(),
                d_init=dS if s["init"] is not None else None)


def _exact_step(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[x].double().repeat_interleave(rep, dim=1) for x in ("q", "k"))
    state, at = s["state"].double(), s["index"].long()
    S = state[at] * torch.exp(s["g"].double())[..., None, None]
    u = s["beta"].double()[..., None] * (s["v"].double() - torch.einsum("bhpn,bhn->bhp", S, k))
    S = S + torch.einsum("bhp,bhn->bhpn", u, k)
    state[at] = S
    return dict(o=s["scale"] * torch.einsum("bhpn,bhn->bhp", S, q), state=state)


def _exact_norm(s):
    h = s["x"].double() + s["residual"].double()
    f = h.to(s["x"].dtype).double()  # the stream as it is kept is what is normalised
    y = f / torch.sqrt((f * f).mean(-1, keepdim=True) + s["eps"]) * s["weight"].double()
    if s["out"] == "same":
        return dict(y=y, stream=h)
    parts = y.reshape(y.shape[0], -1, s["group"] or y.shape[1])
    scale = parts.abs().amax(-1) / E4M3_MAX
    return dict(y8=(parts / scale[..., None]).view_as(y), scale=scale, stream=h)


def _exact_norm_bwd(s):
    h, dy, w = s["x"].double(), s["dy"].double(), s["weight"].double()
    D = h.shape[1]
    n = torch.sqrt((h * h).sum(-1, keepdim=True) / D + s["eps"])
    u = h / n
    t = dy * w
    dx = s["d_stream"].double() + (t - u * ((t * u).sum(-1, keepdim=True) / D)) / n
    return dict(dx=dx, dweight=(dy * u).sum(0))


def exact(case, seed):
    if case["op"] in ("delta_fwd", "delta_bwd"):
        # one step costs some launches and passes over the states: keep it to seconds
        per = case["b"] * case["H"] * case["P"] * case["N"]
        cost = case["L"] * (60e-6 + per * 8 * 8 / 3e12) * (1 if case["op"] == "delta_fwd" else 6)
        if cost > 18.0:
            return None
    s = prepare(case, seed)
    return {"delta_fwd": _exact_delta_fwd, "delta_bwd": _exact_delta_bwd, "step": _exact_step, "norm": _exact_norm,
            "norm_bwd": _exact_norm_bwd}[case["op"]](s)
