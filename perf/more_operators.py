"""Cases and plain forms of the short causal convolution, the selective state
space scan and dropout from a counter-based generator.

Short causal convolution, every channel by itself, K taps (K - 1 inputs in
front of the sequence are the state, xe = [state, x]):

    p_t = bias + sum_k w[:, k] xe_{t+k},   y_t = p_t sigmoid(p_t)

Selective scan, N states a channel, d = softplus(dt + dt_bias):

    h_t = exp(d_t A) h_{t-1} + d_t x_t B_t
    y_t = (C_t . h_t + D x_t) z_t sigmoid(z_t)

Dropout: word j of Philox 4x32-10 with the key `seed` and the counter (block,
offset) decides value 4 block + j of x in row-major order: it is dropped where
the word is below p 2^32, kept values are scaled by 1 / (1 - p), and a residual
is added.

Operators: "conv" (a prompt, from a state or without one, with the final
state), "conv_train" (forward and backward pass through autograd), "conv_step"
(one token), "scan", "scan_train", "scan_step" (the same of the scan),
"dropout" (forward and backward pass with a residual).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, B, S, D, N, dtype, state=False):
    return {"name": name, "op": op, "B": B, "S": S, "D": D, "N": N, "dtype": dtype, "state": state}


def listed():
    """N is the number of states of a channel for the scan, of taps for the convolution."""
    return [
        # the convolution in front of one short float32 sequence: the launch is what counts
        _case("conv_f32_s256_d64", "conv", 1, 256, 64, 4, "f32"),
        # a training step on a ragged batch: odd batch and length, channels of 5 heads of 192
        _case("conv_train_ragged_s1777", "conv_train", 3, 1777, 960, 4, "bf16", True),
        # a training step on the channels of 8 heads of 512
        _case("conv_train_7b_s8192", "conv_train", 8, 8192, 4096, 4, "bf16"),
        # one token of every sequence of a serving batch
        _case("conv_step_7b", "conv_step", 8, 1, 4096, 4, "bf16", True),
        # one short float32 sequence of few channels: the chain of tokens is what counts
        _case("scan_f32_s256_d64", "scan", 1, 256, 64, 16, "f32"),
        # a batch of prompts
        _case("scan_7b_s8192", "scan", 8, 8192, 4096, 16, "bf16"),
        # one long document continued from a state: few channels for the chip, many tokens in a row
        _case("scan_7b_s65536", "scan", 1, 65536, 4096, 16, "bf16", True),
        # a training step on a ragged batch
        _case("scan_train_ragged_s1777", "scan_train", 3, 1777, 960, 16, "bf16", True),
        # a training step on a batch of long sequences
        _case("scan_train_7b_s8192", "scan_train", 8, 8192, 4096, 16, "bf16"),
        # one token of every sequence of a serving batch
        _case("scan_step_7b", "scan_step", 8, 1, 4096, 16, "bf16", True),
        # dropout and the residual sum behind a block, a ragged float32 batch
        _case("dropout_ragged_s1777", "dropout", 3, 1777, 960, 0, "f32"),
        # the same on a batch of long sequences
        _case("dropout_7b_s8192", "dropout", 8, 8192, 4096, 0, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_train", "scan_step", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = _log(rng, 32, 6144)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    B = _log(rng, 1, 64 if op.endswith("step") else 12)
    S = 1 if op.endswith("step") else _log(rng, 1, 16384)
    N = 0 if op == "dropout" else rng.choice([2, 3, 4, 4]) if op.startswith("conv") else rng.choice([16, 16, 16, 32, 64])
    state = op.endswith("step") or (op != "dropout" and rng.random() < 0.5)
    # no more than the largest listed case, and half of it in float32
    most = 8 * 8192 * 4096 * 16 // (1 if dtype == "bf16" else 2)
    S = max(1, min(S, most // (B * D * max(N, 16))))
    return {"op": op, "B": B, "S": S, "D": D, "N": N, "dtype": dtype, "state": state}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, B, S, D, N, t = case["op"], case["B"], case["S"], case["D"], case["N"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda")

    st = dict(case)
    rows = (B, D) if op.endswith("step") else (B, S, D)
    if op == "dropout":
        st["x"], st["r"], st["dy"] = normal(*rows).to(t), normal(*rows).to(t), normal(*rows).to(t)
        st["p"], st["seed"], st["offset"] = 0.1, 2 ** 40 * seed + 12345, 7 * seed
        st["leaves"] = [st[n].requires_grad_(True) for n in ("x", "r")]
        return st
    if op.startswith("conv"):
        st["x"] = normal(*rows).to(t)
        st["w"], st["b"] = uniform(-0.5, 0.5, D, N), uniform(-0.5, 0.5, D)
        st["s0"] = normal(B, N - 1, D).to(t) if case["state"] else None
        if op == "conv_step":
            st["s_out"] = torch.empty_like(st["s0"])
        if op == "conv_train":
            st["dy"] = normal(*rows).to(t)
            st["leaves"] = [st[n].requires_grad_(True) for n in ("x", "w", "b", "s0") if st[n] is not None]
        return st
    # x and the gate are what a convolution and a projection leave; the gate is half of that projection's columns, and
    # B and C are the last columns of the one that the step's rank comes from
    st["x"] = torch.nn.functional.silu(normal(*rows)).to(t)
    st["dt"] = (0.5 * normal(*rows)).to(t)
    st["z"] = normal(*rows[:-1], 2 * D).to(t)[..., D:]
    bc = normal(*rows[:-1], max(1, D // 16) + 2 * N).to(t)
    st["Bm"], st["Cm"] = bc[..., -2 * N:-N], bc[..., -N:]
    # decays: states 1 .. N, steps of 0.001 to 0.1
    st["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * normal(D, N))
    step = torch.exp(uniform(math.log(1e-3), math.log(0.1), D))
    st["bias"] = step + torch.log(-torch.expm1(-step))
    st["Dm"] = 1.0 + 0.1 * normal(D)
    st["h0"] = 0.3 * normal(B, D, N) if case["state"] else None
    if op == "scan_step":
        st["h_out"] = torch.empty_like(st["h0"])
    if op == "scan_train":
        st["dy"] = normal(*rows).to(t)
        for n in ("z", "Bm", "Cm"):
            st[n] = st[n].detach()
        st["leaves"] = [st[n].requires_grad_(True) for n in ("x", "dt", "A", "Bm", "Cm", "Dm", "z", "bias", "h0")
                        if st[n] is not None]
    return st


# ---------------------------------------------------------------------------
# the framework's calls

def _own(st):
    import xlstm_mlstm_chunkwise_amd as mt
    op = st["op"]
    if op == "conv":
        y, s = mt.causal_conv_fw(st["x"], st["w"], st["b"], st["s0"], activation="silu")
        return {"y": y, "s": s}
    if op == "conv_step":
        y, s = mt.causal_conv_step(st["x"], st["w"], st["b"], st["s0"], activation="silu", state_out=st["s_out"])
        return {"y": y, "s": s}
    if op == "conv_train":
        y = mt.causal_conv(st["x"], st["w"], st["b"], st["s0"], activation="silu")
        grads = torch.autograd.grad(y, st["leaves"], st["dy"])
        return {"y": y.detach(), **dict(zip(("dx", "dw", "db", "ds0"), grads))}
    if op == "dropout":
        y = mt.dropout(st["x"], st["p"], st["seed"] % 2 ** 64, st["offset"] % 2 ** 64, residual=st["r"])
        dx, dr = torch.autograd.grad(y, st["leaves"], st["dy"])
        return {"y": y.detach(), "dx": dx, "dr": dr}
    args = [st[n] for n in ("x", "dt", "A", "Bm", "Cm", "Dm", "z", "bias", "h0")]
    if op == "scan":
        y, h = mt.selective_scan_fw(*args)
        return {"y": y, "h": h}
    if op == "scan_step":
        y, h = mt.selective_scan_step(*args, h_out=st["h_out"])
        return {"y": y, "h": h}
    y = mt.selective_scan(*args)
    grads = torch.autograd.grad(y, st["leaves"], st["dy"])
    return {"y": y.detach(), **dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0"), grads))}


# ---------------------------------------------------------------------------
# the plain forms, in float32

def _f(x):
    return x.detach().float()


def _plain_conv(st):
    """p, the extended input and the final state."""
    D, K, S = st["D"], st["N"], st["S"]
    x = st["x"].detach()
    x = x[:, None] if st["op"] == "conv_step" else x
    s0 = x.new_zeros(st["B"], K - 1, D) if st["s0"] is None else st["s0"].detach()
    xe = torch.cat([s0, x], 1)
    w = st["w"].detach()
    p = st["b"].detach() + sum(w[:, k] * xe[:, k:k + S].float() for k in range(K))
    return p, xe, xe[:, S:].contiguous()


def _plain_conv_train(st):
    p, xe, _ = _plain_conv(st)
    K, S, t = st["N"], st["S"], st["x"].dtype
    sig, w = torch.sigmoid(p), st["w"].detach()
    gp = _f(st["dy"]) * sig * (1 + p * (1 - sig))
    dxe = torch.zeros(xe.shape, device=xe.device)
    for k in range(K):
        dxe[:, k:k + S] += w[:, k] * gp
    out = {"y": (p * sig).to(t), "dx": dxe[:, K - 1:].to(t),
           "dw": torch.stack([(gp * xe[:, k:k + S].float()).sum((0, 1)) for k in range(K)], 1), "db": gp.sum((0, 1))}
    if st["s0"] is not None:
        out["ds0"] = dxe[:, :K - 1].to(t)
    return out


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _length(S):
    """Tokens of a chunk: the walks take two steps a token of a chunk, and one a chunk."""
    return 2 ** max(0, round(math.log2(S / 2) / 2)) if S > 2 else S


def _chunks(x, L):
    """(B, S, ...) -> (L, B, chunks, ...) in float32, zeros behind the sequence."""
    x = _f(x)
    pad = -x.shape[1] % L
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
    return x.reshape(x.shape[0], -1, L, *x.shape[2:]).movedim(2, 0)


def _rows(x, S):
    """Inverse of _chunks."""
    x = x.movedim(0, 2)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :S]


def _plain_scan(st, keep):
    """Chunks side by side: the state that a chunk leaves by itself, the states in front of the chunks, then the tokens."""
    S, A = st["S"], st["A"].detach()
    L = _length(S)
    x, Bm, Cm = (_chunks(st[n], L) for n in ("x", "Bm", "Cm"))
    d = _softplus(_f(st["dt"]) + st["bias"].detach())
    d = _chunks(d, L)
    h = torch.zeros(*d.shape[1:], st["N"], device=d.device)
    for i in range(L):
        h = torch.exp(d[i][..., None] * A) * h + (d[i] * x[i])[..., None] * Bm[i][:, :, None]
    total = torch.exp(d.sum(0)[..., None] * A)
    now = torch.zeros_like(h[:, 0]) if st["h0"] is None else st["h0"].detach()
    starts = []
    for c in range(h.shape[1]):
        starts.append(now)
        now = total[:, c] * now + h[:, c]
    h = torch.stack(starts, 1)
    ys, hs = [], [h]
    for i in range(L):
        h = torch.exp(d[i][..., None] * A) * h + (d[i] * x[i])[..., None] * Bm[i][:, :, None]
        ys.append((h * Cm[i][:, :, None]).sum(-1))
        if keep:
            hs.append(h)
    r = _rows(torch.stack(ys), S) + st["Dm"].detach() * _f(st["x"])
    return r, now, (L, x, Bm, Cm, d, hs)


def _plain_scan_train(st):
    S, t, A, z, dy = st["S"], st["x"].dtype, st["A"].detach(), _f(st["z"]), _f(st["dy"])
    r, _, (L, x, Bm, Cm, d, hs) = _plain_scan(st, True)
    sig = torch.sigmoid(z)
    dr = dy * z * sig
    out = {"y": (r * z * sig).to(t)}
    dz = (dy * r * sig * (1 + z * (1 - sig))).to(t)
    gr = _chunks(dr, L)
    # the state gradient that a chunk hands to the one before it, by itself, and with those behind it
    g = torch.zeros_like(hs[0])
    for i in reversed(range(L)):
        g = torch.exp(d[i][..., None] * A) * (g + gr[i][..., None] * Cm[i][:, :, None])
    total = torch.exp(d.sum(0)[..., None] * A)
    now, ends = torch.zeros_like(g[:, 0]), [None] * g.shape[1]
    for c in reversed(range(g.shape[1])):
        ends[c] = now
        now = total[:, c] * now + g[:, c]
    g = torch.stack(ends, 1)
    dx, dd, dB, dC, dA = [None] * L, [None] * L, [None] * L, [None] * L, torch.zeros_like(A)
    for i in reversed(range(L)):
        g = g + gr[i][..., None] * Cm[i][:, :, None]
        dC[i] = (gr[i][..., None] * hs.pop()).sum(2)
        dB[i] = (g * (d[i] * x[i])[..., None]).sum(2)
        s = (g * Bm[i][:, :, None]).sum(-1)
        g = torch.exp(d[i][..., None] * A) * g
        w = g * hs[-1]
        dA += (d[i][..., None] * w).sum((0, 1))
        dd[i] = x[i] * s + (w * A).sum(-1)
        dx[i] = d[i] * s
    ddt = _rows(torch.stack(dd), S) * torch.sigmoid(_f(st["dt"]) + st["bias"].detach())
    out["dx"] = (_rows(torch.stack(dx), S) + st["Dm"].detach() * dr).to(t)
    out["ddt"], out["dA"] = ddt.to(t), dA
    out["dB"], out["dC"] = _rows(torch.stack(dB), S).to(t), _rows(torch.stack(dC), S).to(t)
    out["dD"], out["dz"], out["dbias"] = (dr * _f(st["x"])).sum((0, 1)), dz, ddt.sum((0, 1))
    if st["h0"] is not None:
        out["dh0"] = now
    return out


def _plain_scan_step(st):
    x, z, Bm, Cm = (_f(st[n]) for n in ("x", "z", "Bm", "Cm"))
    d = _softplus(_f(st["dt"]) + st["bias"])
    h = torch.exp(d[..., None] * st["A"]) * st["h0"] + (d * x)[..., None] * Bm[:, None]
    r = (h * Cm[:, None]).sum(-1) + st["Dm"] * x
    return (r * z * torch.sigmoid(z)).to(st["x"].dtype), h


def _kept(n, p, seed, offset, device):
    """The generator's decisions for n values, true where a value is kept: 32-bit words in int64."""
    low, blocks = 0xFFFFFFFF, -(-n // 4)
    i = torch.arange(blocks, device=device)
    c = [i & low, i >> 32, torch.full_like(i, offset & low), torch.full_like(i, (offset >> 32) & low)]
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        m0, m1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]   # the product's 64 bits, whatever the sign
        c = [((m1 >> 32) & low) ^ c[1] ^ k0, m1 & low, ((m0 >> 32) & low) ^ c[3] ^ k1, m0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return (torch.stack(c, 1) >= int(p * 2 ** 32)).flatten()[:n]


def _plain_dropout(st):
    x, t = st["x"].detach(), st["x"].dtype
    kept = _kept(x.numel(), st["p"], st["seed"], st["offset"], x.device).view(x.shape)
    scale = 1 / (1 - st["p"])
    y = torch.where(kept, x.float() * scale, 0.0) + _f(st["r"])
    return {"y": y.to(t), "dx": torch.where(kept, _f(st["dy"]) * scale, 0.0).to(t), "dr": st["dy"]}


def run(st):
    if own:
        return _own(st)
    op, t = st["op"], st["x"].dtype
    if op == "dropout":
        return _plain_dropout(st)
    if op == "conv_train":
        return _plain_conv_train(st)
    if op.startswith("conv"):
        p, _, s = _plain_conv(st)
        y = (p * torch.sigmoid(p)).to(t)
        return {"y": y[:, 0] if op == "conv_step" else y, "s": s}
    if op == "scan_train":
        return _plain_scan_train(st)
    if op == "scan_step":
        y, h = _plain_scan_step(st)
        return {"y": y, "h": h}
    r, h, _ = _plain_scan(st, False)
    z = _f(st["z"])
    return {"y": (r * z * torch.sigmoid(z)).to(t), "h": h}


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op, B, S, D, N = case["op"], case["B"], case["S"], case["D"], case["N"]
    size = 2 if case["dtype"] == "bf16" else 4
    rows = B * S * D
    if op == "dropout":
        # x, residual and dy in; y and dx out (the residual's gradient is dy itself)
        return {"bytes": 5 * rows * size, "flops": 3.0 * rows}
    if op.startswith("conv"):
        state, weight = B * (N - 1) * D * size, 4 * D * (N + 1)
        if op == "conv_train":
            # x and dy in, y and dx out, the weights and their gradients
            return {"bytes": 4 * rows * size + 2 * weight + (2 * state if case["state"] else 0), "flops": (6.0 * N + 12) * rows}
        return {"bytes": 2 * rows * size + weight + state * (2 if case["state"] else 1), "flops": (2.0 * N + 4) * rows}
    state, weight, cols = 4 * B * D * N, 4 * D * (N + 2), 2 * B * S * N * size
    if op == "scan_train":
        # x, dt, z, dy, B, C in; y, dx, ddt, dz, dB, dC out; weights and their gradients.  A state and token: the
        # forward's product, exponential and two sums, six products and sums of the gradients behind them
        return {"bytes": 8 * rows * size + 2 * cols + 2 * weight + (2 * state if case["state"] else 0), "flops": 22.0 * rows * N}
    return {"bytes": 4 * rows * size + cols + weight + state * (2 if case["state"] else 1), "flops": 7.0 * rows * N}


# ---------------------------------------------------------------------------
# the definitions in 64 bits: token by token

def _exact_conv(case, st):
    K, S = case["N"], case["S"]
    x, w, b = st["x"].detach().double(), st["w"].detach().double(), st["b"].detach().double()
    x = x[:, None] if case["op"] == "conv_step" else x
    s0 = torch.zeros(case["B"], K - 1, case["D"], dtype=torch.float64, device=x.device) if st["s0"] is None else st["s0"].detach().double()
    windows = torch.cat([s0, x], 1).unfold(1, K, 1)              # (B, S, D, K)
    p = (windows * w).sum(-1) + b
    e = torch.exp(-p)
    y = p / (1 + e)
    if case["op"] != "conv_train":
        last = torch.cat([s0, x], 1)[:, S:]
        return {"y": y[:, 0] if case["op"] == "conv_step" else y, "s": last}
    g = st["dy"].double() * ((1 + e) + p * e) / (1 + e) ** 2
    # an input's gradient: the K outputs that saw it, the last tap first
    ge = torch.nn.functional.pad(g, (0, 0, K - 1, K - 1)).unfold(1, K, 1)
    dxe = (ge * w.flip(1)).sum(-1)
    out = {"y": y, "dx": dxe[:, K - 1:], "dw": (g[..., None] * windows).sum((0, 1)), "db": g.sum((0, 1))}
    if st["s0"] is not None:
        out["ds0"] = dxe[:, :K - 1]
    return out


def _exact_scan(case, st):
    names = ("x", "dt", "z", "Bm", "Cm", "A", "Dm", "bias")
    x, dt, z, Bm, Cm, A, Dm, bias = (st[n].detach().double() for n in names)
    step = case["op"] == "scan_step"
    if step:
        x, dt, z, Bm, Cm = (v[:, None] for v in (x, dt, z, Bm, Cm))
    S = x.shape[1]
    d = torch.logaddexp(dt + bias, torch.zeros((), dtype=torch.float64, device=x.device))
    h = torch.zeros(case["B"], case["D"], case["N"], dtype=torch.float64, device=x.device) if st["h0"] is None else st["h0"].detach().double()

    def advance(h, t):
        h = torch.exp(d[:, t, :, None] * A).mul_(h)
        return h.addcmul_((d[:, t] * x[:, t])[..., None], Bm[:, t, None])

    r = torch.empty_like(x)
    stretch, starts = 64, []
    for t in range(S):
        if t % stretch == 0 and case["op"] == "scan_train":
            starts.append(h.clone())
        h = advance(h, t)
        r[:, t] = torch.matmul(h, Cm[:, t, :, None])[..., 0]
    r += Dm * x
    gate = z / (1 + torch.exp(-z))
    if case["op"] != "scan_train":
        y = r * gate
        return {"y": y[:, 0] if step else y, "h": h}
    dy = st["dy"].double()
    dr = dy * gate
    out = {"y": r * gate}
    dz = dy * r * (1 + torch.exp(-z) * (1 + z)) / (1 + torch.exp(-z)) ** 2
    dx, dd, dB, dC, dA = torch.empty_like(x), torch.empty_like(x), torch.empty_like(Bm), torch.empty_like(Cm), torch.zeros_like(A)
    g = torch.zeros_like(h)
    for j in reversed(range(len(starts))):
        hs = [starts.pop()]
        for t in range(j * stretch, min(S, (j + 1) * stretch)):
            hs.append(advance(hs[-1], t))
        for t in reversed(range(j * stretch, min(S, (j + 1) * stretch))):
            g = g.addcmul_(dr[:, t, :, None], Cm[:, t, None])
            dC[:, t] = torch.matmul(dr[:, t, None], hs.pop())[:, 0]
            dB[:, t] = torch.matmul((d[:, t] * x[:, t])[:, None], g)[:, 0]
            du = torch.matmul(g, Bm[:, t, :, None])[..., 0]
            g = g * torch.exp(d[:, t, :, None] * A)
            de = g * hs[-1]                                       # the gradient of d A
            dA += torch.einsum("bd,bdn->dn", d[:, t], de)
            dd[:, t] = du * x[:, t] + (de * A).sum(-1)
            dx[:, t] = du * d[:, t]
    ddt = dd * torch.sigmoid(dt + bias)
    out.update(dx=dx + Dm * dr, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dr * x).sum((0, 1)), dz=dz, dbias=ddt.sum((0, 1)))
    if st["h0"] is not None:
        out["dh0"] = g
    return out


def _exact_words(blocks, seed, offset, device):
    """Philox 4x32-10 in 16-bit limbs: every product and sum stays below 2^63."""
    def mulhilo(m, c):
        mh, ml, ch, cl = m >> 16, m & 0xFFFF, c >> 16, c & 0xFFFF
        mid = mh * cl + (ml * cl >> 16)
        mid2 = ml * ch + (mid & 0xFFFF)
        return mh * ch + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (ml * cl & 0xFFFF)

    i = torch.arange(blocks, device=device)
    w = [i % 2 ** 32, i // 2 ** 32, torch.full_like(i, offset % 2 ** 32), torch.full_like(i, offset // 2 ** 32 % 2 ** 32)]
    for n in range(10):
        key = (seed % 2 ** 32 + n * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + n * 0xBB67AE85) % 2 ** 32
        h0, l0 = mulhilo(0xD2511F53, w[0])
        h1, l1 = mulhilo(0xCD9E8D57, w[2])
        w = [h1 ^ w[1] ^ key[0], l1, h0 ^ w[3] ^ key[1], l0]
    return torch.stack(w, -1).flatten()


def _exact_dropout(case, st):
    x, n = st["x"].detach(), st["x"].numel()
    dropped = (_exact_words((n + 3) // 4, st["seed"], st["offset"], x.device)[:n] < math.floor(st["p"] * 4294967296)).view(x.shape)
    q = 1 - st["p"]
    y = (x.double() / q).masked_fill(dropped, 0.0) + st["r"].detach().double()
    return {"y": y, "dx": (st["dy"].double() / q).masked_fill(dropped, 0.0), "dr": st["dy"].double()}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "dropout":
        return _exact_dropout(case, st)
    return (_exact_conv if case["op"].startswith("conv") else _exact_scan)(case, st)
