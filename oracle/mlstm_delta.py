"""Float64 oracle of the gated delta rule and of the head norm: the definition
token by token, its adjoint recurrence, and the norm's formulas.  It shares no
code with the GPU path and uses no chunks.

Per head, with a_t = sigmoid(f_t), b_t = sigmoid(i_t):

    r_t = v_t - a_t C_{t-1}^T k_t,   u_t = b_t r_t
    C_t = a_t C_{t-1} + k_t u_t^T,   h_t = s C_t^T q_t

Arrays have any leading axes, then (S, D) for q, k, v and (S,) for the gates.
"""
from __future__ import annotations

import numpy as np


def _sigmoid(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def _prepare(q, k, v, i_pre, f_pre, C0, qk_scale):
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    C = np.zeros(q.shape[:-2] + (q.shape[-1], v.shape[-1])) if C0 is None else np.array(C0, np.float64)
    s = 1.0 / np.sqrt(q.shape[-1]) if qk_scale is None or qk_scale <= 0 else float(qk_scale)
    return q, k, v, _sigmoid(f_pre), _sigmoid(i_pre), C, s


def _t(C, x):
    """C^T x over the leading axes."""
    return np.matmul(x[..., None, :], C)[..., 0, :]


def delta_fw(q, k, v, i_pre, f_pre, C0=None, qk_scale=None):
    """(H, C): the recurrence token by token."""
    q, k, v, a, b, C, s = _prepare(q, k, v, i_pre, f_pre, C0, qk_scale)
    H = np.empty(v.shape)
    for t in range(q.shape[-2]):
        at, kt = a[..., t, None], k[..., t, :]
        u = b[..., t, None] * (v[..., t, :] - at * _t(C, kt))
        C = at[..., None] * C + kt[..., :, None] * u[..., None, :]
        H[..., t, :] = s * _t(C, q[..., t, :])
    return H, C


def delta_grad(q, k, v, i_pre, f_pre, dH, C0=None, dC=None, qk_scale=None):
    """Gradients of sum(dH * H) + sum(dC * C) by the adjoint recurrence, as a
    dict with dQ, dK, dV, d_i, d_f, dC0."""
    q, k, v, a, b, C, s = _prepare(q, k, v, i_pre, f_pre, C0, qk_scale)
    S = q.shape[-2]
    states, rs = [C], []
    for t in range(S):
        at, kt = a[..., t, None], k[..., t, :]
        rs.append(v[..., t, :] - at * _t(C, kt))
        C = at[..., None] * C + kt[..., :, None] * (b[..., t, None] * rs[-1])[..., None, :]
        states.append(C)
    dH = np.asarray(dH, np.float64)
    G = np.zeros_like(C) if dC is None else np.array(dC, np.float64)
    dq, dk, dv, da, db = (np.empty_like(x) for x in (q, k, v, a, b))
    for t in reversed(range(S)):
        C, before, r = states[t + 1], states[t], rs[t]
        at, kt, bt, dh = a[..., t, None], k[..., t, :], b[..., t, None], dH[..., t, :]
        dq[..., t, :] = s * np.matmul(C, dh[..., None])[..., 0]
        G = G + s * q[..., t, :, None] * dh[..., None, :]
        du = _t(G, kt)
        db[..., t] = (du * r).sum(-1)
        dr = bt * du
        dv[..., t, :] = dr
        dk[..., t, :] = np.matmul(G, (bt * r)[..., None])[..., 0] - at * np.matmul(before, dr[..., None])[..., 0]
        da[..., t] = (G * before).sum((-1, -2)) - (dr * _t(before, kt)).sum(-1)
        G = at[..., None] * (G - kt[..., :, None] * dr[..., None, :])
    # 1 - sigmoid(x) as sigmoid(-x): near 1 the difference keeps no digits, in 64 bits either
    return dict(dQ=dq, dK=dk, dV=dv, d_i=db * b * _sigmoid(-np.asarray(i_pre, np.float64)),
                d_f=da * a * _sigmoid(-np.asarray(f_pre, np.float64)), dC0=G)


def head_norm_fw(x, weight=None, bias=None, eps=1e-6):
    """y (B, S, NH, D) of x (B, NH, S, D)."""
    x = np.asarray(x, np.float64)
    n = (x - x.mean(-1, keepdims=True)) / np.sqrt(x.var(-1, keepdims=True) + eps)
    y = np.swapaxes(n, 1, 2)
    y = y if weight is None else y * np.asarray(weight, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def head_norm_grad(x, dy, weight=None, eps=1e-6):
    """(dx, dweight, dbias) of sum(dy * y)."""
    x, dy = np.asarray(x, np.float64), np.swapaxes(np.asarray(dy, np.float64), 1, 2)
    rstd = 1.0 / np.sqrt(x.var(-1, keepdims=True) + eps)
    n = (x - x.mean(-1, keepdims=True)) * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)[None, :, None, :]
    dx = rstd * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    return dx, (dy * n).sum((0, 2)), dy.sum((0, 2))
