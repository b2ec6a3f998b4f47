"""Float64 oracle of the short causal convolution, the selective scan and
dropout: the definitions token by token and the adjoint recurrence.  It shares
no code with the GPU path and uses no chunks.

    conv:  xe = [state, x],  p_t = bias + sum_k w[:, k] xe_{t+k},  y = p or p sigmoid(p)
    scan:  d = softplus(dt + dt_bias),  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,
           y_t = (C_t . h_t + D x_t) gate_t,  gate = z sigmoid(z) or 1
"""
from __future__ import annotations

import numpy as np


def _f(x):
    return np.asarray(x, np.float64)


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-_f(x)))


def softplus(x):
    x = _f(x)
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def silu(x):
    return _f(x) * _sigmoid(x)


def silu_slope(x):
    s = _sigmoid(x)
    return s * (1.0 + _f(x) * (1.0 - s))


# ---------------------------------------------------------------------------
# convolution: x (B, S, D), w (D, K), state (B, K - 1, D)

def _extended(x, w, state):
    B, S, D = x.shape
    K = w.shape[1]
    state = np.zeros((B, K - 1, D)) if state is None else _f(state)
    return np.concatenate([state, _f(x)], 1)


def conv_fw(x, w, bias=None, state=None, act=True):
    """(y, state')."""
    xe, w, S = _extended(x, w, state), _f(w), x.shape[1]
    p = sum(w[:, k] * xe[:, k:k + S] for k in range(w.shape[1])) + (0.0 if bias is None else _f(bias))
    return (silu(p) if act else p), xe[:, S:]


def conv_grad(x, w, dy, bias=None, state=None, dstate=None, act=True, slope=None):
    """Gradients of sum(dy * y) + sum(dstate * state') as a dict with dx, dw, db,
    dstate.  slope replaces the activation's."""
    xe, w, S, K = _extended(x, w, state), _f(w), x.shape[1], w.shape[1]
    p = sum(w[:, k] * xe[:, k:k + S] for k in range(K)) + (0.0 if bias is None else _f(bias))
    g = _f(dy) * ((silu_slope(p) if act else 1.0) if slope is None else slope)
    dxe = np.zeros(xe.shape)
    for k in range(K):
        dxe[:, k:k + S] += w[:, k] * g
    if dstate is not None:
        dxe[:, S:] += _f(dstate)
    dw = np.stack([(g * xe[:, k:k + S]).sum((0, 1)) for k in range(K)], 1)
    return dict(dx=dxe[:, K - 1:], dw=dw, db=g.sum((0, 1)), dstate=dxe[:, :K - 1])


# ---------------------------------------------------------------------------
# scan: x, d, gate (B, S, D), a (B, S, D, N), B, C (B, S, N)

def scan_walk(d, a, x, Bm, Cm, D, gate, h0):
    """(y, h, states): the recurrence with the steps d, the decays a and the gate
    given; states[t] is the state in front of token t."""
    h, states, r = h0, [h0], []
    for t in range(x.shape[1]):
        h = a[:, t] * h + (d[:, t] * x[:, t])[..., None] * Bm[:, t, None]
        states.append(h)
        r.append((h * Cm[:, t, None]).sum(-1) + D * x[:, t])
    r = np.stack(r, 1) if r else np.zeros(x.shape)
    return r * gate, h, states, r


def scan_walk_grad(d, a, x, Bm, Cm, A, D, gate, slope, dy, h0, dh):
    """The adjoint recurrence; slope is the gate's derivative.  dd is the
    gradient of the steps."""
    _, _, states, r = scan_walk(d, a, x, Bm, Cm, D, gate, h0)
    dr = dy * gate
    g, dA = np.array(dh, np.float64), np.zeros(A.shape)
    dx, dd, dB, dC = np.zeros(x.shape), np.zeros(x.shape), np.zeros(Bm.shape), np.zeros(Cm.shape)
    for t in reversed(range(x.shape[1])):
        g = g + dr[:, t, :, None] * Cm[:, t, None]
        dC[:, t] = (dr[:, t, :, None] * states[t + 1]).sum(1)
        dB[:, t] = (g * (d[:, t] * x[:, t])[..., None]).sum(1)
        s = (g * Bm[:, t, None]).sum(-1)
        g = a[:, t] * g
        w = g * states[t]
        dA += (d[:, t, :, None] * w).sum(0)
        dd[:, t] = x[:, t] * s + (A * w).sum(-1)
        dx[:, t] = d[:, t] * s + D * dr[:, t]
    return dict(dx=dx, dd=dd, dA=dA, dB=dB, dC=dC, dD=(dr * x).sum((0, 1)), dz=dy * r * slope, dh0=g)


def _prepare(x, dt, A, Bm, Cm, D, z, dt_bias, h0):
    x, dt, A, Bm, Cm = (_f(v) for v in (x, dt, A, Bm, Cm))
    D = np.zeros(x.shape[-1]) if D is None else _f(D)
    pre = dt + (0.0 if dt_bias is None else _f(dt_bias))
    d = softplus(pre)
    h0 = np.zeros((x.shape[0],) + A.shape) if h0 is None else _f(h0)
    gate = np.ones(x.shape) if z is None else silu(z)
    return d, np.exp(d[..., None] * A), x, Bm, Cm, A, D, gate, pre, h0


def scan_fw(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None):
    """(y, h)."""
    d, a, x, Bm, Cm, A, D, gate, _, h0 = _prepare(x, dt, A, Bm, Cm, D, z, dt_bias, h0)
    return scan_walk(d, a, x, Bm, Cm, D, gate, h0)[:2]


def scan_grad(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, h0=None, dh=None):
    """Gradients of sum(dy * y) + sum(dh * h) as a dict with dx, ddt, dA, dB, dC,
    dD, dz, dbias, dh0."""
    d, a, x, Bm, Cm, A, D, gate, pre, h0 = _prepare(x, dt, A, Bm, Cm, D, z, dt_bias, h0)
    slope = np.zeros(x.shape) if z is None else silu_slope(z)
    g = scan_walk_grad(d, a, x, Bm, Cm, A, D, gate, slope, _f(dy), h0, np.zeros(h0.shape) if dh is None else _f(dh))
    g["ddt"] = g.pop("dd") * _sigmoid(pre)
    g["dbias"] = g["ddt"].sum((0, 1))
    return g


# ---------------------------------------------------------------------------
# dropout

def philox_words(blocks, seed, offset):
    """Words of Philox 4x32 with ten rounds for the counters (block, offset) and
    the key seed, (len(blocks), 4) uint32."""
    low = np.uint64(0xFFFFFFFF)
    i = np.asarray(blocks, np.uint64)
    off = np.uint64(offset % 2 ** 64)
    c = [i & low, i >> np.uint64(32), np.broadcast_to(off & low, i.shape), np.broadcast_to(off >> np.uint64(32), i.shape)]
    k = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
    for _ in range(10):
        m0, m1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(m1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), m1 & low, (m0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), m0 & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, -1).astype(np.uint32)


def kept(n, p, seed, offset=0):
    """Which of n values dropout keeps."""
    words = philox_words(np.arange((n + 3) // 4), seed, offset).ravel()[:n]
    return words.astype(np.float64) >= np.floor(p * 2.0 ** 32)


def dropout(x, p, seed, offset=0, residual=None):
    y = np.where(kept(np.size(x), p, seed, offset).reshape(np.shape(x)), _f(x) / (1.0 - p), 0.0)
    return y if residual is None else y + _f(residual)
