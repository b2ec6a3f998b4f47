"""Cases and plain forms of the gated delta rule and the head norm.

The gated delta rule is the matrix-memory recurrence of the sigmoid-input-gate
cell with a correction by what the memory already returns for the key.  Per
head, with a_t = sigmoid(f_t), b_t = sigmoid(i_t), s = 1 / sqrt(DHQK):

    u_t = b_t (v_t - a_t C_{t-1}^T k_t)
    C_t = a_t C_{t-1} + k_t u_t^T
    h_t = s C_t^T q_t

The head norm is the layer norm of every row of H over its DHV values, with a
weight and a bias per head and channel; it reads (B, NH, S, D) and writes
(B, S, NH, D), the layout of the projection behind it.

Operators: "fw" (a prompt or a forward pass from a state, with the final
state), "train" (forward and backward pass through autograd), "step" (one
token for every head), "norm" (the head norm), "norm_train" (the head norm
and its backward pass, weight and bias gradients included).
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, B, NH, S, DK, DV, dtype, state=False):
    return {"name": name, "op": op, "B": B, "NH": NH, "S": S, "DK": DK, "DV": DV, "dtype": dtype, "state": state}


def listed():
    return [
        # one short sequence of one float32 head: the launches and their order are what counts
        _case("fw_f32_s256_d64", "fw", 1, 1, 256, 64, 64, "f32"),
        # a batch of prompts on 7B-shaped heads
        _case("fw_7b_s8192", "fw", 8, 8, 8192, 256, 512, "bf16"),
        # one long document continued from a state: few heads, many chunks in a row
        _case("fw_7b_s65536", "fw", 1, 8, 65536, 256, 512, "bf16", True),
        # a training step on a ragged batch: odd batch and heads, a length that ends inside a chunk
        _case("train_ragged_s1777", "train", 3, 5, 1777, 64, 192, "bf16", True),
        # a training step on medium heads
        _case("train_s2048_d128", "train", 8, 8, 2048, 128, 128, "bf16"),
        # a training step on 7B-shaped heads
        _case("train_7b_s8192", "train", 8, 8, 8192, 256, 512, "bf16"),
        # one token of one small sequence: latency alone
        _case("step_f32_d64", "step", 1, 4, 1, 64, 64, "f32", True),
        # one token of every sequence of a serving batch on 7B-shaped heads
        _case("step_7b", "step", 8, 8, 1, 256, 512, "bf16", True),
        # the norm behind that token
        _case("norm_decode", "norm", 8, 8, 1, 0, 512, "f32"),
        # the norm behind a batch of prompts
        _case("norm_7b_s8192", "norm", 8, 8, 8192, 0, 512, "bf16"),
        # the norm in a training step on a ragged batch, float32 H as the cell gives it by default
        _case("norm_train_ragged", "norm_train", 3, 5, 1777, 0, 192, "f32"),
        # the norm in a training step on 7B-shaped heads
        _case("norm_train_7b", "norm_train", 8, 8, 8192, 0, 512, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fw", "train", "step", "norm", "norm_train"])
    B, NH = _log(rng, 1, 12), _log(rng, 1, 16)
    DK, DV = rng.choice([64, 128, 256]), 64 * rng.randint(1, 8)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    state = rng.random() < 0.5
    if op == "step":
        S = 1
    elif op == "fw":
        S = _log(rng, 1, 16384)
    else:
        S = _log(rng, 1, 8192)
    if op.startswith("norm"):
        DK, state = 0, False
    # no more than the largest listed case, and half of it in float32
    most = 8 * 8 * 8192 * 256 * 512 // (1 if dtype == "bf16" else 2)
    S = max(1, min(S, most // (B * NH * max(DK, 64) * DV)))
    return {"op": op, "B": B, "NH": NH, "S": S, "DK": DK, "DV": DV, "dtype": dtype, "state": state}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, NH, S, DK, DV, t = case["B"], case["NH"], case["S"], case["DK"], case["DV"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda")

    st = dict(case)
    if case["op"].startswith("norm"):
        # H comes with a scale of its own in every row, and a mean
        st["x"] = ((normal(B, NH, S, DV) + 0.3) * uniform(0.1, 2.0, B, NH, S, 1)).to(t)
        st["w"], st["b"] = 1.0 + 0.2 * normal(NH, DV), 0.1 * normal(NH, DV)
        if case["op"] == "norm_train":
            st["dy"] = normal(B, S, NH, DV).to(torch.bfloat16)
            st["leaves"] = [st[n].requires_grad_(True) for n in ("x", "w", "b")]
        return st
    rows = (B, NH) if case["op"] == "step" else (B, NH, S)
    k = normal(*rows, DK)
    # keys of unit length, as the rule needs them (b_t |k_t|^2 < 2)
    k /= k.norm(dim=-1, keepdim=True)
    st["q"], st["k"], st["v"] = normal(*rows, DK).to(t), k.to(t), normal(*rows, DV).to(t)
    st["i"], st["f"] = normal(*rows), uniform(2.0, 6.0, *rows)
    st["C0"] = 0.1 * normal(B, NH, DK, DV) if case["state"] else None
    if case["op"] == "step":
        st["C_out"] = torch.empty(B, NH, DK, DV, device="cuda")
    if case["op"] == "train":
        st["dH"] = normal(B, NH, S, DV).to(t)
        st["leaves"] = [st[n].requires_grad_(True) for n in ("q", "k", "v", "i", "f", "C0") if st[n] is not None]
    return st


# ---------------------------------------------------------------------------
# the framework's calls

def _own(st):
    import xlstm_mlstm_chunkwise_amd as mt
    op = st["op"]
    if op == "fw":
        H, C = mt.mlstm_delta_fw(st["q"], st["k"], st["v"], st["i"], st["f"], st["C0"], h_dtype=TYPES[st["dtype"]])
        return {"H": H, "C": C}
    if op == "step":
        h, C = mt.mlstm_delta_step(st["q"], st["k"], st["v"], st["i"], st["f"], st["C0"], C_out=st["C_out"],
                                   h_dtype=TYPES[st["dtype"]])
        return {"h": h, "C": C}
    if op == "train":
        H = mt.mlstm_delta(st["q"], st["k"], st["v"], st["i"], st["f"], st["C0"], h_dtype=TYPES[st["dtype"]])
        grads = torch.autograd.grad(H, st["leaves"], st["dH"])
        return {"H": H.detach(), **dict(zip(("dq", "dk", "dv", "di", "df", "dC0"), grads))}
    if op == "norm":
        return {"y": mt.head_norm_fw(st["x"], st["w"], st["b"], eps=EPS, y_dtype=torch.bfloat16)}
    y = mt.head_norm(st["x"], st["w"], st["b"], eps=EPS, y_dtype=torch.bfloat16)
    dx, dw, db = torch.autograd.grad(y, st["leaves"], st["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw, "db": db}


# ---------------------------------------------------------------------------
# the plain form: chunks of 64 tokens in float32, every head at once

def _chunks(x, n, pad):
    """(B, NH, S, ...) -> (n, B, NH, CHUNK, ...) in float32, zeros behind the sequence."""
    x = x.detach().float()
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[:2] + (pad,) + x.shape[3:])], 2)
    return x.reshape(x.shape[:2] + (n, CHUNK) + x.shape[3:]).movedim(2, 0)


def _rows(x, S):
    """Inverse of _chunks."""
    x = x.movedim(0, 2)
    return x.reshape(x.shape[:2] + (-1,) + x.shape[4:])[:, :, :S]


def _unit_inverse(A):
    """(I + A)^-1 of strictly lower triangular A (.., CHUNK, CHUNK): diagonal blocks of twice the size each time."""
    T = torch.eye(CHUNK, device=A.device).expand(A.shape).contiguous()
    size = 1
    while size < CHUNK:
        pairs = CHUNK // (2 * size)
        t, a = (x.reshape(x.shape[:-2] + (pairs, 2 * size, pairs, 2 * size)) for x in (T, A))
        at = torch.arange(pairs, device=A.device)
        t, a = t[..., at, :, at, :], a[..., at, :, at, :]          # (pairs, .., 2 size, 2 size)
        low = -(t[..., size:, size:] @ a[..., size:, :size] @ t[..., :size, :size])
        T.reshape(T.shape[:-2] + (pairs, 2 * size, pairs, 2 * size))[..., at, size:, at, :size] = low
        size *= 2
    return T


def _plain_chunks(st):
    """What every chunk needs before the states are known."""
    S = st["S"]
    n = -(-S // CHUNK)
    pad = n * CHUNK - S
    q, k, v = (_chunks(st[x], n, pad) for x in ("q", "k", "v"))
    i, f = (_chunks(st[x], n, pad) for x in ("i", "f"))
    beta, lf = torch.sigmoid(i), torch.nn.functional.logsigmoid(f)
    if pad:
        beta[-1, :, :, CHUNK - pad:] = 0
        lf[-1, :, :, CHUNK - pad:] = 0
    b = torch.cumsum(lf, -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~low, -math.inf))
    A = (beta[..., None] * D * (k @ k.mT)).tril(-1)
    T = _unit_inverse(A) * beta[..., None, :]
    P = D * (q @ k.mT)
    return q, k, v, beta, b, D, T, P


def _plain_forward(st):
    """H in float32, the final state, and what the backward pass reads."""
    q, k, v, beta, b, D, T, P = _plain_chunks(st)
    s = st["DK"] ** -0.5
    C = torch.zeros(st["B"], st["NH"], st["DK"], st["DV"], device=q.device) if st["C0"] is None else st["C0"].detach()
    e, w, last = torch.exp(b)[..., None], torch.exp(b[..., -1:] - b)[..., None], torch.exp(b[..., -1])[..., None, None]
    states, us = [], []
    for c in range(q.shape[0]):
        u = T[c] @ (v[c] - e[c] * (k[c] @ C))
        states.append(C)
        us.append(u)
        C = last[c] * C + k[c].mT @ (w[c] * u)
    states, u = torch.stack(states), torch.stack(us)
    H = s * (e * (q @ states) + P @ u)
    return _rows(H, st["S"]), C, (q, k, v, beta, b, D, T, P, states, u, e, w, last)


def _plain_step(st):
    q, k, v = (st[x].float() for x in ("q", "k", "v"))
    a, beta = torch.sigmoid(st["f"])[..., None], torch.sigmoid(st["i"])[..., None]
    C = st["C0"] if st["C0"] is not None else torch.zeros_like(st["C_out"])
    u = beta * (v - a * (k[..., None, :] @ C)[..., 0, :])
    C = a[..., None] * C + k[..., :, None] * u[..., None, :]
    return (st["DK"] ** -0.5) * (q[..., None, :] @ C)[..., 0, :], C


def _plain_train(st):
    S, s = st["S"], st["DK"] ** -0.5
    H, C, (q, k, v, beta, b, D, T, P, states, u, e, w, last) = _plain_forward(st)
    n = q.shape[0]
    dh = s * _chunks(st["dH"], n, n * CHUNK - S)
    dC = torch.zeros_like(C)
    dus, dCs = [None] * n, [None] * n
    for c in reversed(range(n)):
        dCs[c] = dC
        r = T[c].mT @ (P[c].mT @ dh[c] + w[c] * (k[c] @ dC))   # the gradient of v
        dus[c] = r
        dC = last[c] * dC + q[c].mT @ (e[c] * dh[c]) - k[c].mT @ (e[c] * r)
    dv, dCs = torch.stack(dus), torch.stack(dCs)
    after = torch.cat([states[1:], C[None]])
    dP = D * (dh @ u.mT)
    dG = -(D * (dv @ u.mT)).tril(-1)
    dq = e * (dh @ states.mT) + dP @ k
    dk = dP.mT @ q + (dG + dG.mT) @ k - e * (dv @ states.mT) + w * (u @ dCs.mT)
    di = (1 - beta) * (dv / beta.clamp(min=1e-30)[..., None] * u).sum(-1)
    db = (q * dq).sum(-1) - (v * dv).sum(-1)
    db[..., -1] += (after * dCs).sum((-1, -2))
    dlf = torch.cumsum(db.flip(-1), -1).flip(-1)
    df = _rows(dlf, S) * torch.sigmoid(-st["f"].detach())
    t = st["q"].dtype
    out = {"H": H.to(t), "dq": _rows(dq, S).to(t), "dk": _rows(dk, S).to(t), "dv": _rows(dv, S).to(t), "di": _rows(di, S), "df": df}
    if st["C0"] is not None:
        out["dC0"] = dC
    return out


def _plain_norm(x, w, b):
    x = x.detach().float()
    d = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n = (d * r).transpose(1, 2)                               # (B, S, NH, D)
    return n, r.transpose(1, 2), n * w.detach() + b.detach()


def run(st):
    if own:
        return _own(st)
    op = st["op"]
    if op == "fw":
        H, C, _ = _plain_forward(st)
        return {"H": H.to(st["q"].dtype), "C": C}
    if op == "step":
        h, C = _plain_step(st)
        return {"h": h.to(st["q"].dtype), "C": C}
    if op == "train":
        return _plain_train(st)
    n, r, y = _plain_norm(st["x"], st["w"], st["b"])
    if op == "norm":
        return {"y": y.to(torch.bfloat16).contiguous()}
    dy = st["dy"].float()
    g = dy * st["w"].detach()
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    return {"y": y.to(torch.bfloat16).contiguous(), "dx": dx.transpose(1, 2).contiguous().to(st["x"].dtype),
            "dw": (dy * n).sum((0, 1)), "db": dy.sum((0, 1))}


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    B, NH, S, DK, DV = case["B"], case["NH"], case["S"], case["DK"], case["DV"]
    size = 2 if case["dtype"] == "bf16" else 4
    rows = B * NH * S
    if case["op"].startswith("norm"):
        if case["op"] == "norm":
            return {"bytes": rows * DV * (size + 2) + 8 * NH * DV, "flops": 8.0 * rows * DV}
        # x and dy in; y and dx out; weight, bias and their gradients
        return {"bytes": rows * DV * (2 * size + 4) + 16 * NH * DV, "flops": 20.0 * rows * DV}
    state = 4 * B * NH * DK * DV
    inputs = rows * ((2 * DK + DV) * size + 8) + (state if case["state"] else 0)
    if case["op"] == "train":
        # the forward's three products with the state, and six of the gradients; H, dH and every gradient
        return {"bytes": 2 * inputs + 2 * rows * DV * size, "flops": 18.0 * rows * DK * DV}
    return {"bytes": inputs + rows * DV * size + state, "flops": 6.0 * rows * DK * DV}


# ---------------------------------------------------------------------------
# the definition in 64 bits: the recurrence token by token

def _exact_train(st, q, k, v, a, beta, C):
    """Forward, then the adjoint recurrence backwards; the states of a stretch of tokens are formed again from its start."""
    B, NH, S, DK, DV = st["B"], st["NH"], st["S"], st["DK"], st["DV"]
    s, stretch = DK ** -0.5, 64
    H = torch.empty(B, NH, S, DV, dtype=torch.float64, device=q.device)
    starts = []
    for t in range(S):
        if t % stretch == 0:
            starts.append(C)
        u = beta[:, :, t, None] * (v[:, :, t] - a[:, :, t, None] * torch.einsum("bhkv,bhk->bhv", C, k[:, :, t]))
        C = a[:, :, t, None, None] * C + k[:, :, t, :, None] * u[:, :, None, :]
        H[:, :, t] = s * torch.einsum("bhkv,bhk->bhv", C, q[:, :, t])
    dh = st["dH"].double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    da, dbeta = torch.empty_like(a), torch.empty_like(beta)
    G = torch.zeros_like(C)
    for j in reversed(range(len(starts))):
        C, before, rs, us = starts.pop(), [], [], []
        for t in range(j * stretch, min(S, (j + 1) * stretch)):
            before.append(C)
            rs.append(v[:, :, t] - a[:, :, t, None] * torch.einsum("bhkv,bhk->bhv", C, k[:, :, t]))
            us.append(beta[:, :, t, None] * rs[-1])
            C = a[:, :, t, None, None] * C + k[:, :, t, :, None] * us[-1][:, :, None, :]
        for t in reversed(range(j * stretch, min(S, (j + 1) * stretch))):
            C0, r, u = before.pop(), rs.pop(), us.pop()
            dq[:, :, t] = s * torch.einsum("bhkv,bhv->bhk", C, dh[:, :, t])
            G = G + s * q[:, :, t, :, None] * dh[:, :, t, None, :]
            du = torch.einsum("bhkv,bhk->bhv", G, k[:, :, t])
            dbeta[:, :, t] = (du * r).sum(-1)
            dv[:, :, t] = beta[:, :, t, None] * du
            at, Ck = a[:, :, t, None], torch.einsum("bhkv,bhk->bhv", C0, k[:, :, t])
            dk[:, :, t] = torch.einsum("bhkv,bhv->bhk", G, u) - at * torch.einsum("bhkv,bhv->bhk", C0, dv[:, :, t])
            da[:, :, t] = (G * C0).sum((-1, -2)) - (dv[:, :, t] * Ck).sum(-1)
            G = at[..., None] * (G - k[:, :, t, :, None] * dv[:, :, t, None, :])
            C = C0
    out = {"H": H, "dq": dq, "dk": dk, "dv": dv, "di": dbeta * beta * (1 - beta), "df": da * a * torch.sigmoid(-st["f"].detach().double())}
    if st["C0"] is not None:
        out["dC0"] = G
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        x = st["x"].detach().double().permute(0, 2, 1, 3)
        w, b = st["w"].detach().double(), st["b"].detach().double()
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        sd = torch.sqrt(var + EPS)
        y = (x - mean) / sd * w + b
        if case["op"] == "norm":
            return {"y": y}
        dy = st["dy"].double()
        # the derivative of (x - mean) / sd along dy w, term by term
        g = dy * w / sd
        dvar = -0.5 * (g * (x - mean)).sum(-1, keepdim=True) / (var + EPS)
        dx = g - g.mean(-1, keepdim=True) + 2 * dvar * (x - mean) / case["DV"]
        return {"y": y, "dx": dx.permute(0, 2, 1, 3).contiguous(), "dw": torch.einsum("bshd,bshd->hd", dy, (x - mean) / sd),
                "db": torch.einsum("bshd->hd", dy)}
    q, k, v = (st[n].detach().double() for n in ("q", "k", "v"))
    a, beta = torch.sigmoid(st["f"].detach().double()), torch.sigmoid(st["i"].detach().double())
    B, NH, S, DK, DV = case["B"], case["NH"], case["S"], case["DK"], case["DV"]
    C = torch.zeros(B, NH, DK, DV, dtype=torch.float64, device=q.device) if st["C0"] is None else st["C0"].detach().double()
    if case["op"] == "train":
        return _exact_train(st, q, k, v, a, beta, C)
    if case["op"] == "step":
        q, k, v, a, beta = (x[:, :, None] for x in (q, k, v, a, beta))
    H = torch.empty(B, NH, S, DV, dtype=torch.float64, device=q.device)
    for t in range(S):
        u = beta[:, :, t, None] * (v[:, :, t] - a[:, :, t, None] * torch.einsum("bhkv,bhk->bhv", C, k[:, :, t]))
        C = torch.addcmul(a[:, :, t, None, None] * C, k[:, :, t, :, None], u[:, :, None, :])
        H[:, :, t] = (DK ** -0.5) * torch.einsum("bhkv,bhk->bhv", C, q[:, :, t])
    if case["op"] == "step":
        return {"h": H[:, :, 0], "C": C}
    return {"H": H, "C": C}
