"""Oracle: gated delta rule and row norm (test infrastructure only).

The fast weight of oracle/ttt_linear.py with the squared binding loss: after a
decay by a_t = exp(g_t), one gradient step of size beta_t on
    l_t(W) = 1/2 |W k_t - v_t|^2,   grad = (W k_t - v_t) k_t^T,
so with S = W^T [dk, dv]
    e_t = v_t - a_t S_{t-1}^T k_t,  S_t = a_t S_{t-1} + beta_t k_t e_t^T,  o_t = scale S_t^T q_t.
All arithmetic is float64.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def delta_recurrent(q, k, v, g, beta, S0=None, scale=None, keep=False):
    """q, k: [B,H,N,dk]; v: [B,H,N,dv]; g (None: no decay), beta: [B,H,N];
    S0: [B,H,dk,dv] or None.  Returns (out, S_end); keep: also every state
    (N + 1 of them) and every e."""
    q, k, v, beta = _f64(q), _f64(k), _f64(v), _f64(beta)
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    scale = dk ** -0.5 if scale is None or scale <= 0 else scale
    a = np.ones((B, H, N)) if g is None else np.exp(_f64(g))
    S = np.zeros((B, H, dk, dv)) if S0 is None else _f64(S0).copy()
    out, es, states = np.empty((B, H, N, dv)), np.empty((B, H, N, dv)), [S]
    for t in range(N):
        S = a[:, :, t, None, None] * S
        e = v[:, :, t] - np.einsum("bhij,bhi->bhj", S, k[:, :, t])
        S = S + beta[:, :, t, None, None] * (k[:, :, t, :, None] * e[:, :, None, :])
        out[:, :, t] = scale * np.einsum("bhij,bhi->bhj", S, q[:, :, t])
        es[:, :, t] = e
        if keep:
            states.append(S)
    return (out, S, states, es) if keep else (out, S)


def delta_backward(q, k, v, g, beta, dout, S0=None, dS_end=None, scale=None):
    """Gradients of sum <dout, out> + <dS_end, S_end>: (dq, dk, dv, dg, dbeta,
    dS0), dg None where g is.  The reverse-time recurrence of the definition."""
    _, _, S, es = delta_recurrent(q, k, v, g, beta, S0, scale, keep=True)
    q, k, v, beta, dout = _f64(q), _f64(k), _f64(v), _f64(beta), _f64(dout)
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    scale = dk ** -0.5 if scale is None or scale <= 0 else scale
    a = np.ones((B, H, N)) if g is None else np.exp(_f64(g))
    X = np.zeros((B, H, dk, dv)) if dS_end is None else _f64(dS_end).copy()
    gq, gk, gv = np.empty(q.shape), np.empty(k.shape), np.empty(v.shape)
    gg, gb = np.empty(beta.shape), np.empty(beta.shape)
    for t in range(N - 1, -1, -1):
        do, kt, bt = dout[:, :, t], k[:, :, t], beta[:, :, t, None]
        X = X + scale * q[:, :, t, :, None] * do[:, :, None, :]
        gq[:, :, t] = scale * np.einsum("bhij,bhj->bhi", S[t + 1], do)
        du = np.einsum("bhij,bhi->bhj", X, kt)
        gv[:, :, t] = bt * du
        gb[:, :, t] = (du * es[:, :, t]).sum(-1)
        decayed = a[:, :, t, None, None] * S[t]
        gk[:, :, t] = bt * (np.einsum("bhij,bhj->bhi", X, es[:, :, t])
                            - np.einsum("bhij,bhj->bhi", decayed, du))
        Y = X - kt[..., :, None] * (bt * du)[..., None, :]
        gg[:, :, t] = (Y * decayed).sum((-1, -2))
        X = a[:, :, t, None, None] * Y
    return gq, gk, gv, (None if g is None else gg), gb, X


def _act(z, gate):
    s = 1 / (1 + np.exp(-z))
    return (s, s * (1 - s)) if gate == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def _rstd(x, kind, eps):
    ss = (x * x).sum(-1, keepdims=True)
    return 1 / np.sqrt(ss / x.shape[-1] + eps) if kind == "rms" else 1 / np.maximum(np.sqrt(ss), eps)


def row_norm(x, w=None, z=None, res=None, kind="rms", gate="none", eps=1e-6, scale=1.0):
    """out = res + scale * x r(x) * w * act(z), row by row."""
    x = _f64(x)
    y = scale * x * _rstd(x, kind, eps)
    if w is not None:
        y = y * _f64(w)
    if gate != "none":
        y = y * _act(_f64(z), gate)[0]
    return y if res is None else y + _f64(res)


def row_norm_backward(x, dout, w=None, z=None, kind="rms", gate="none", eps=1e-6, scale=1.0):
    """(dx, dw, dz) of sum <dout, row_norm(x, ...)>; None where the input is."""
    x, p = _f64(x), scale * _f64(dout)
    r = _rstd(x, kind, eps)
    n = x * r
    wv = np.ones(x.shape[-1]) if w is None else _f64(w)
    dz = None
    if gate != "none":
        act, dact = _act(_f64(z), gate)
        dz = p * n * wv * dact
        p = p * act
    dw = None if w is None else (p * n).reshape(-1, x.shape[-1]).sum(0)
    dn = p * wv
    proj = n * (dn * n).sum(-1, keepdims=True) / (x.shape[-1] if kind == "rms" else 1)
    if kind == "l2":   # below eps the factor is a constant
        proj = np.where(np.sqrt((x * x).sum(-1, keepdims=True)) > eps, proj, 0.0)
    return r * (dn - proj), dw, dz
