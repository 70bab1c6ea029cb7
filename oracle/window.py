"""fp64 oracle of window attention (include/window.h), of the exit norm (include/norm.h)
and of the scan's one-token step: plain NumPy from the definitions, token by token.

Test infrastructure only.  Pinned by tests/test_oracle_window.py to differences and special cases."""
import numpy as np


def seen(t, window, sinks):
    """The tokens that token t sees."""
    s = np.arange(t + 1)
    return s[(t - s < window) | (s < sinks)]


def _valid(valid_len, b, L):
    return np.full(b, L) if valid_len is None else np.clip(np.asarray(valid_len), 0, L)


def window_forward(q, k, v, window, sinks, scale, valid_len=None):
    """(o [b, L, H, P], lse [b, H, L]) of q [b, L, H, P] and k, v [b, L, G, P]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    b, L, H, P = q.shape
    G = k.shape[2]
    o, lse = np.zeros((b, L, H, P)), np.zeros((b, H, L))
    for i, V in enumerate(_valid(valid_len, b, L)):
        for t in range(V):
            s = seen(t, window, sinks)
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                x = scale * q[i, t, hs] @ k[i, s, g].T
                m = x.max(-1, keepdims=True)
                e = np.exp(x - m)
                o[i, t, hs] = e @ v[i, s, g] / e.sum(-1, keepdims=True)
                lse[i, hs, t] = m[:, 0] + np.log(e.sum(-1))
    return o, lse


def window_backward(q, k, v, do, window, sinks, scale, valid_len=None, o=None):
    """dict(dq, dk, dv) for the gradient do of o.  With `o`, do . o takes that in place of the exact outputs, as a kernel does
    that is given outputs as they were stored."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    o = None if o is None else np.asarray(o, np.float64)
    b, L, H, P = q.shape
    G = k.shape[2]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for i, V in enumerate(_valid(valid_len, b, L)):
        for t in range(V):
            s = seen(t, window, sinks)
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                x = scale * q[i, t, hs] @ k[i, s, g].T
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                dp = do[i, t, hs] @ v[i, s, g].T
                D = (p * dp).sum(-1, keepdims=True) if o is None else (do[i, t, hs] * o[i, t, hs]).sum(-1, keepdims=True)
                dx = scale * p * (dp - D)
                dq[i, t, hs] = dx @ k[i, s, g]
                dk[i, s, g] += dx.T @ q[i, t, hs]
                dv[i, s, g] += p.T @ do[i, t, hs]
    return dict(dq=dq, dk=dk, dv=dv)


def rounding_of_o(q, k, v, do, window, sinks, scale, valid_len=None):
    """Bounds (dq, dk) on what the gradients' rows move by when do . o takes an o whose elements are off by half a
    bf16 step, 2^-8 of them: the norms of scale sum_s p_ts k_s and of scale sum_t p_ts q_t times 2^-8 sum_i |do_i o_i|."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    b, L, H, P = q.shape
    G = k.shape[2]
    dq, dk = np.zeros((b, L, H)), np.zeros((b, L, G))
    for i, V in enumerate(_valid(valid_len, b, L)):
        for t in range(V):
            s = seen(t, window, sinks)
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                x = scale * q[i, t, hs] @ k[i, s, g].T
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                off = abs(scale) * 2.0 ** -8 * np.abs(do[i, t, hs] * (p @ v[i, s, g])).sum(-1)
                dq[i, t, hs] = off * np.linalg.norm(p @ k[i, s, g], axis=-1)
                dk[i, s, g] += (off * np.linalg.norm(q[i, t, hs], axis=-1)) @ p
    return dict(dq=dq, dk=dk)


def entry(t, window, sinks):
    """Where token t lies in a ring."""
    return t if t < sinks else sinks + (t - sinks) % window


def window_fill(x, cache, window, sinks, valid_len=None, index=None):
    """The ring `cache` [slots, sinks + window, G, P] after the prompts x [b, L, G, P]: token by token."""
    cache = np.array(cache)
    b, L = x.shape[:2]
    for i, V in enumerate(_valid(valid_len, b, L)):
        slot = i if index is None else int(index[i])
        if 0 <= slot < cache.shape[0]:
            for t in range(V):
                cache[slot, entry(t, window, sinks)] = x[i, t]
    return cache


def window_step(q, k, v, k_cache, v_cache, position, window, sinks, scale, index=None):
    """(o [b, H, P], k_cache, v_cache) after one token of every request."""
    q, k_cache, v_cache = np.asarray(q, np.float64), np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    b, H, P = q.shape
    G = k.shape[1]
    o = np.zeros_like(q)
    for i in range(b):
        slot, t = (i if index is None else int(index[i])), int(position[i])
        if t < 0 or not 0 <= slot < k_cache.shape[0]:
            continue
        k_cache[slot, entry(t, window, sinks)], v_cache[slot, entry(t, window, sinks)] = k[i], v[i]
        n = min(t + 1, sinks + window)
        for h in range(H):
            g = h // (H // G)
            x = scale * k_cache[slot, :n, g] @ q[i, h]
            e = np.exp(x - x.max())
            o[i, h] = e @ v_cache[slot, :n, g] / e.sum()
    return o, k_cache, v_cache


def _act(name, z):
    """The activation and its derivative."""
    s = 1 / (1 + np.exp(-z))
    return {None: (z, np.ones_like(z)), "silu": (z * s, s + z * s * (1 - s)), "sigmoid": (s, s * (1 - s))}[name]


def group_norm(x, weight, bias, gate, groups, eps, center, activation, gate_first, dy=None):
    """y [rows, D], and with dy also dict(dx, dgate, dweight, dbias)."""
    x = np.asarray(x, np.float64)
    R, D = x.shape
    w = D // groups
    a, da = (None, None) if gate is None else _act(activation, np.asarray(gate, np.float64))
    u = (x * a if gate_first else x).reshape(R, groups, w)
    if center:
        u = u - u.mean(-1, keepdims=True)
    r = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    n = (u * r).reshape(R, D)
    y = n * weight + (0.0 if bias is None else bias)
    if gate is None:
        out, slope = _act(activation, y)
    else:
        out = y if gate_first else y * a
    if dy is None:
        return out
    dy = np.asarray(dy, np.float64)
    g = dy * slope if gate is None else (dy if gate_first else dy * a)
    t = (g * weight).reshape(R, groups, w)
    ng = n.reshape(R, groups, w)
    du = r * (t - ng * (t * ng).mean(-1, keepdims=True) - (t.mean(-1, keepdims=True) if center else 0.0))
    du = du.reshape(R, D)
    dgate = None if gate is None else (du * x * da if gate_first else dy * y * da)
    return out, dict(dx=du * a if gate_first else du, dgate=dgate, dweight=(g * n).sum(0), dbias=g.sum(0))


def ssd_step(x, dt, A, B, C, D, state, index=None):
    """(y [b, H, P], state) after one token of every request."""
    state = np.array(state, np.float64)
    b, H, P = x.shape
    G = B.shape[1]
    y = np.zeros((b, H, P))
    for i in range(b):
        slot = i if index is None else int(index[i])
        if not 0 <= slot < state.shape[0]:
            continue
        for h in range(H):
            g = h // (H // G)
            S = np.exp(float(dt[i, h]) * float(A[h])) * state[slot, h] + float(dt[i, h]) * np.outer(x[i, h], B[i, g]).astype(np.float64)
            state[slot, h] = S
            y[i, h] = S @ C[i, g] + D[h] * x[i, h]
    return y, state
