"""The short causal convolution, the cells, the norm and dropout as a block uses
them: in a row, one token after another, through autograd, captured, on other
streams (needs an MI355X)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import conv_fw, dropout, scan_fw  # noqa: E402
from oracle.mlstm_block import silu  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _weights(seed, M, D, N, R, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = dict(up=n(M, 2 * D) / M ** 0.5, conv=0.5 * n(D, 4), conv_b=0.1 * n(D), cols=n(D, R + 2 * N) / D ** 0.5, dt=n(R, D) / R ** 0.5,
             A=-torch.exp(0.5 * n(D, N)), D=1 + 0.1 * n(D), dt_bias=-2 + 0.5 * n(D), down=n(D, M) / D ** 0.5)
    return {k: v.to(dtype) if k in ("up", "cols", "dt", "down") else v for k, v in w.items()}


def _block(mt, x, w, N, R, p=0.0, seed=1, offset=0, state=None, keep_state=False):
    """A block with the scan as its cell: projections, convolution, scan with its
    gate, projection, dropout and the residual sum."""
    D = w["conv"].shape[0]
    xz = x @ w["up"]
    s0, h0 = state if state is not None else (None, None)
    if keep_state:
        xc, s = mt.causal_conv_fw(xz[..., :D], w["conv"], w["conv_b"], s0, activation="silu")
        cols = xc @ w["cols"]
        y, h = mt.selective_scan_fw(xc, cols[..., :R] @ w["dt"], w["A"], cols[..., R:R + N], cols[..., R + N:], w["D"], xz[..., D:],
                                    w["dt_bias"], h0)
        return mt.dropout_fw((y @ w["down"]), p, seed, offset, residual=x), (s, h)
    xc = mt.causal_conv(xz[..., :D], w["conv"], w["conv_b"], s0, activation="silu")
    cols = xc @ w["cols"]
    y = mt.selective_scan(xc, cols[..., :R] @ w["dt"], w["A"], cols[..., R:R + N], cols[..., R + N:], w["D"], xz[..., D:], w["dt_bias"], h0)
    return mt.dropout(y @ w["down"], p, seed, offset, residual=x)


def _reference(x, w, N, R, p, seed, offset):
    """The same in float64 on the host."""
    w = {k: v.detach().double().cpu().numpy() for k, v in w.items()}
    x = x.detach().double().cpu().numpy()
    D = w["conv"].shape[0]
    xz = x @ w["up"]
    xc, _ = conv_fw(xz[..., :D], w["conv"], w["conv_b"])
    cols = xc @ w["cols"]
    y, _ = scan_fw(xc, cols[..., :R] @ w["dt"], w["A"], cols[..., R:R + N], cols[..., R + N:], w["D"], xz[..., D:], w["dt_bias"])
    return dropout(y @ w["down"], p, seed, offset, x)


def test_a_block_and_its_gradients(mt):
    """Against float64: five float32 operators in a row, each off by less than
    2^-18 of its magnitudes here; and the gradients of every weight against
    central differences of the float64 block (step 1e-6, off by 1e-9)."""
    M, D, N, R = 24, 40, 16, 4
    w = {k: v.requires_grad_(True) for k, v in _weights(1, M, D, N, R).items()}
    x = torch.randn(2, 37, M, device="cuda", requires_grad=True)
    y = _block(mt, x, w, N, R, 0.2, 11, 12)
    ref = _reference(x, w, N, R, 0.2, 11, 12)
    assert np.abs(y.detach().double().cpu().numpy() - ref).max() < 5 * 2.0 ** -18 * np.abs(ref).max()
    dy = torch.randn_like(y)
    grads = torch.autograd.grad(y, [x, *w.values()], dy)
    rng = np.random.default_rng(3)
    for name, g in zip(("x", *w), grads):
        d = rng.standard_normal(g.shape)
        d /= np.linalg.norm(d)
        ends = []
        for s in (1e-6, -1e-6):
            step = torch.from_numpy(s * d).cuda()
            moved = {k: v.detach().double() + (step if k == name else 0) for k, v in w.items()}
            ends.append((dy.double().cpu().numpy() * _reference(x.detach().double() + (step if name == "x" else 0), moved, N, R, 0.2, 11, 12)).sum())
        diff, got = (ends[0] - ends[1]) / 2e-6, (g.double().cpu().numpy() * d).sum()
        assert abs(diff - got) < 1e-4 * max(1.0, float(g.double().norm())), name


def test_prompt_then_tokens(mt):
    """A prompt, then one token at a time from its states: the rows of one pass
    over all of them, to float32's rounding."""
    M, D, N, R = 16, 72, 16, 3
    w = _weights(5, M, D, N, R)
    x = torch.randn(3, 30, M, device="cuda")
    whole, _ = _block(mt, x, w, N, R, keep_state=True)
    y, (s, h) = _block(mt, x[:, :21].contiguous(), w, N, R, keep_state=True)
    rows = [y]
    for t in range(21, 30):
        xz = x[:, t] @ w["up"]
        xc, s = mt.causal_conv_step(xz[:, :D], w["conv"], w["conv_b"], s, activation="silu", state_out=s)
        cols = xc @ w["cols"]
        yt, h = mt.selective_scan_step(xc, cols[:, :R] @ w["dt"], w["A"], cols[:, R:R + N], cols[:, R + N:], w["D"], xz[:, D:], w["dt_bias"], h,
                                       h_out=h)
        rows.append((x[:, t] + yt @ w["down"])[:, None])
    assert (torch.cat(rows, 1) - whole).abs().max() < 2.0 ** -16 * whole.abs().max()


def test_in_front_of_the_matrix_memory(mt):
    """Convolution, gated delta rule, norm, dropout and residual: the cell of this
    library with the operators around it, forward and backward."""
    B, S, NH, DK, DV = 2, 70, 2, 64, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = n(B, S, NH * DK).requires_grad_(True)
    w, wn = (0.5 * n(NH * DK, 4)).requires_grad_(True), (1 + 0.1 * n(NH, DV)).requires_grad_(True)
    i, f = n(B, NH, S), 3 + n(B, NH, S)
    xc = mt.causal_conv(x, w, activation="silu")
    heads = lambda v: v.view(B, S, NH, DK).transpose(1, 2).contiguous()
    k = torch.nn.functional.normalize(heads(xc), dim=-1)
    y = mt.mlstm_delta(heads(xc), k, heads(x), i, f, norm_weight=wn).reshape(B, S, NH * DV)
    out = mt.dropout(y, 0.1, 3, 4, residual=x)
    loss = out.square().sum()
    grads = torch.autograd.grad(loss, [x, w, wn])
    assert all(torch.isfinite(v).all() and v.abs().sum() > 0 for v in grads)
    kept = mt.dropout_fw(torch.ones_like(y), 0.1, 3, 4) > 0
    assert torch.equal(out[~kept], x.detach()[~kept])


def test_captured_and_replayed(mt):
    """A training pass of the block in one graph, replayed with new inputs and a
    new seed between eager passes: the eager bits."""
    M, D, N, R = 16, 48, 16, 2
    w = {k: v.requires_grad_(True) for k, v in _weights(9, M, D, N, R, torch.float32).items()}
    # the library's own operators only: their leaves are what a projection gives
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    shapes = dict(x=(2, 50, D), dt=(2, 50, D), z=(2, 50, D), Bm=(2, 50, N), Cm=(2, 50, N), res=(2, 50, D), dy=(2, 50, D))
    io = {k: n(*s) for k, s in shapes.items()}
    seed = torch.tensor([1, 2], device="cuda")

    def work():
        xc, s = mt.causal_conv_fw(io["x"], w["conv"].detach(), w["conv_b"].detach(), activation="silu")
        y, h = mt.selective_scan_fw(xc, io["dt"], w["A"].detach(), io["Bm"], io["Cm"], w["D"].detach(), io["z"], w["dt_bias"].detach())
        out = mt.dropout_fw(y, 0.1, seed, residual=io["res"])
        dy = mt.dropout_fw(io["dy"], 0.1, seed)
        r = mt.selective_scan_bw(xc, io["dt"], w["A"].detach(), io["Bm"], io["Cm"], dy, w["D"].detach(), io["z"], w["dt_bias"].detach())
        c = mt.causal_conv_bw(io["x"], w["conv"].detach(), r["dx"], w["conv_b"].detach(), activation="silu")
        hs, _ = mt.selective_scan_step(io["x"][:, 0], io["dt"][:, 0], w["A"].detach(), io["Bm"][:, 0], io["Cm"][:, 0], h=h)
        return [out, s, h, hs] + [r[k] for k in sorted(r)] + [c[k] for k in sorted(c)]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for turn in range(3):
        for v in io.values():
            v.copy_(n(*v.shape))
        seed.add_(turn + 1)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(got, work()))


def test_a_captured_training_pass(mt):
    """Forward and backward through autograd in one graph, no eager graph of the
    same leaves alive."""
    D, N = 40, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    leaves = [v.requires_grad_(True) for v in (n(1, 33, D), n(D, 4), n(1, 33, D), -torch.exp(n(D, N)), n(1, 33, N), n(1, 33, N))]
    x, cw, dt, A, B, C = leaves
    dy, seed = n(1, 33, D), torch.tensor([5, 6], device="cuda")

    def work():
        xc = mt.causal_conv(x, cw, activation="silu")
        y = mt.dropout(mt.selective_scan(xc, dt, A, B, C), 0.1, seed, residual=x)
        return [y.detach(), *torch.autograd.grad(y, leaves, dy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(3):
        with torch.no_grad():
            for v in leaves[:3]:
                v.copy_(n(*v.shape))
        seed.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(got, work()))


def _two(mt, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    D, N = 200, 16
    x, dt, z, B, C, dy = n(2, 300, D), n(2, 300, D), n(2, 300, D), n(2, 300, N), n(2, 300, N), n(2, 300, D)
    A, w = -torch.exp(n(D, N)), n(D, 4)

    def work(ws=None):
        xc, s = mt.causal_conv_fw(x, w, activation="silu")
        y, h = mt.selective_scan_fw(xc, dt, A, B, C, None, z, workspace=ws)
        y = mt.dropout_fw(y, 0.3, seed)
        r = mt.selective_scan_bw(xc, dt, A, B, C, dy, None, z, workspace=ws)
        c = mt.causal_conv_bw(x, w, r["dx"], activation="silu", workspace=ws)
        return [y, s, h] + [r[k] for k in sorted(r)] + [c[k] for k in sorted(c)]

    return work


def test_two_streams_at_once(mt):
    works = [_two(mt, j) for j in range(2)]
    want = [wk() for wk in works]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((j, works[j]()))
    torch.cuda.synchronize()
    for j, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[j]))


def test_two_graphs_that_share_a_workspace(mt):
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    graphs = []
    for j in range(2):
        work = _two(mt, 10 + j)
        want = [o.clone() for o in work(ws)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = work(ws)
        graphs.append((g, out, want, work))
    for j in (0, 1, 1, 0):
        g, out, want, work = graphs[j]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(graphs[1 - j][3](ws), graphs[1 - j][2]))


def test_gate_of_the_convolution_is_silu(mt):
    x = torch.linspace(-20, 20, 64, device="cuda").view(1, 1, 64)
    y, _ = mt.causal_conv_fw(x, torch.tensor([[0.0, 1.0]], device="cuda").expand(64, 2).contiguous(), activation="silu")
    ref = silu(x.double().cpu().numpy())
    assert np.abs(y.double().cpu().numpy() - ref).max() < 2.0 ** -23 * 70 * 20
