"""The gated delta rule token by token in fp64 (NumPy), its reverse-mode
derivative, and the residual addition with a root-mean-square norm with its
derivative: the definitions in include/delta.h and include/norm.h, for tests."""
import numpy as np


def _heads(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[2], axis=2)


def delta_forward(q, k, v, g, beta, scale, init=None, valid_len=None):
    """o [b, L, H, P] and the final state [b, H, P, N]."""
    b, L, H, P = v.shape
    q, k, v = _heads(q, H), _heads(k, H), np.asarray(v, np.float64)
    a, beta = np.exp(np.asarray(g, np.float64)), np.asarray(beta, np.float64)
    S = np.zeros((b, H, P, k.shape[3])) if init is None else np.array(init, np.float64)
    o = np.zeros(v.shape)
    for i in range(b):
        V = L if valid_len is None else int(np.clip(valid_len[i], 0, L))
        for t in range(V):
            Sd = a[i, :, t, None, None] * S[i]
            z = v[i, t] - np.einsum("hpn,hn->hp", Sd, k[i, t])
            S[i] = Sd + np.einsum("hp,hn->hpn", beta[i, :, t, None] * z, k[i, t])
            o[i, t] = scale * np.einsum("hpn,hn->hp", S[i], q[i, t])
    return o, S


def delta_backward(q, k, v, g, beta, scale, do, d_final=None, init=None, valid_len=None):
    """Gradients of <do, o> + <d_final, final state>."""
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    qh, kh, v, do = _heads(q, H), _heads(k, H), np.asarray(v, np.float64), np.asarray(do, np.float64)
    a, beta = np.exp(np.asarray(g, np.float64)), np.asarray(beta, np.float64)
    S0 = np.zeros((b, H, P, N)) if init is None else np.array(init, np.float64)
    D = np.zeros((b, H, P, N)) if d_final is None else np.array(d_final, np.float64)
    dq, dk, dv = np.zeros(qh.shape), np.zeros(kh.shape), np.zeros(v.shape)
    dg, dbeta = np.zeros(a.shape), np.zeros(a.shape)
    for i in range(b):
        V = L if valid_len is None else int(np.clip(valid_len[i], 0, L))
        S, kept = S0[i], []
        for t in range(V):
            Sd = a[i, :, t, None, None] * S
            z = v[i, t] - np.einsum("hpn,hn->hp", Sd, kh[i, t])
            S = Sd + np.einsum("hp,hn->hpn", beta[i, :, t, None] * z, kh[i, t])
            kept.append((Sd, z, S))
        for t in reversed(range(V)):
            Sd, z, S = kept[t]
            be, x = beta[i, :, t, None], scale * do[i, t]
            dq[i, t] = np.einsum("hp,hpn->hn", x, S)
            D[i] += np.einsum("hp,hn->hpn", x, qh[i, t])
            Dk = np.einsum("hpn,hn->hp", D[i], kh[i, t])
            dbeta[i, :, t] = (Dk * z).sum(-1)
            dz = be * Dk
            dv[i, t] = dz
            dk[i, t] = np.einsum("hp,hpn->hn", be * z, D[i]) - np.einsum("hp,hpn->hn", dz, Sd)
            D[i] -= np.einsum("hp,hn->hpn", dz, kh[i, t])
            dg[i, :, t] = (D[i] * Sd).sum((-1, -2))
            D[i] *= a[i, :, t, None, None]
    per = H // G
    return dict(dq=dq.reshape(b, L, G, per, N).sum(3), dk=dk.reshape(b, L, G, per, N).sum(3), dv=dv, dg=dg, dbeta=dbeta,
                d_init=D)


def delta_step(q, k, v, g, beta, scale, state, index=None):
    """o [b, H, P]; `state` [slots, H, P, N] is updated in place."""
    b, H, _ = v.shape
    index = np.arange(b) if index is None else index
    o = np.zeros(v.shape)
    for i in range(b):
        if not 0 <= index[i] < len(state):
            continue
        oi, S = delta_forward(q[i][None, None], k[i][None, None], v[i][None, None], g[i][None, :, None],
                              beta[i][None, :, None], scale, state[index[i]][None])
        o[i], state[index[i]] = oi[0, 0], S[0]
    return o


def add_rms_norm(stream, weight, eps):
    """y for the stored stream."""
    h = np.asarray(stream, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def add_rms_norm_backward(dy, stream, weight, eps, d_stream=None):
    h, dy, w = (np.asarray(x, np.float64) for x in (stream, dy, weight))
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    t = dy * w
    dx = r * t - h * r ** 3 * (t * h).mean(-1, keepdims=True)
    if d_stream is not None:
        dx = dx + np.asarray(d_stream, np.float64)
    return dx, (dy * h * r).reshape(-1, h.shape[-1]).sum(0)
