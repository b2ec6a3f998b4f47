"""Parity of the gated delta rule (mlstm_delta_fw, _bw, _step and the autograd
function) against the float64 oracle (needs an MI355X).

Inputs are seeded draws, keys of unit length; Q, K, V, dH are rounded to bf16
for the bf16 cases and both sides read the same values.

Tolerances.  Every computed operand carries 24 bits into the matrix cores, so
an output is a chain of at most five products, each a float32 sum of at most
512 terms; a sum of n terms rounds n times by half a step, 2^-24 of the
running sum, independently: sqrt(n) 2^-24.  F32 = 5 sqrt(512) 2^-24 = 6.8e-6 of
the largest magnitude of the tensor.  d_f is a sum over up to 64 rows of
differences of row sums whose terms do not shrink with the result: sqrt(64)
times that.  dQ, dK, dV and H stored as bf16 round by at most 2^-8 of the value;
the terms of dK then have two-part operands, each off by at most 2^-15
(truncation at sixteen bits), three such products in a row: DK_BF16 = 3 * 2^-15
of the largest magnitude on top.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import delta_fw, delta_grad, head_norm_fw, head_norm_grad  # noqa: E402
from workloads import round_to_bf16  # noqa: E402

pytestmark = pytest.mark.gpu

F32 = 5 * np.sqrt(512) * 2.0 ** -24
GATE = 8 * F32
DK_BF16 = 3 * 2.0 ** -15


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def _dtype(kind):
    return torch.bfloat16 if kind == "bf16" else torch.float32


def _draw(seed, B, NH, S, DK, DV, kind, state=True, hkind=None):
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((B, NH, S, DK))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    x = dict(q=rng.standard_normal((B, NH, S, DK)).astype(np.float32), k=k.astype(np.float32),
             v=rng.standard_normal((B, NH, S, DV)).astype(np.float32))
    if kind == "bf16":
        x = {n: round_to_bf16(a)[0] for n, a in x.items()}
    x["i"] = rng.standard_normal((B, NH, S)).astype(np.float32)
    x["f"] = (1.0 + 5.0 * rng.random((B, NH, S))).astype(np.float32)
    x["C0"] = (0.3 * rng.standard_normal((B, NH, DK, DV))).astype(np.float32) if state else None
    x["dH"] = rng.standard_normal((B, NH, S, DV)).astype(np.float32)
    if (hkind or kind) == "bf16":
        x["dH"] = round_to_bf16(x["dH"])[0]
    x["dC"] = rng.standard_normal((B, NH, DK, DV)).astype(np.float32)
    return x


def _gpu(x, kind):
    t = _dtype(kind)
    args = [_dev(x[n], t) for n in ("q", "k", "v")] + [_dev(x[n], torch.float32) for n in ("i", "f")]
    return args, None if x["C0"] is None else _dev(x["C0"], torch.float32)


def _close(got, ref, rel, what, factor=1.0):
    bf16 = got.dtype == torch.bfloat16
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), what
    if not ref.size:
        return
    limit = factor * rel * np.abs(ref).max() + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0)
    over = np.abs(got - ref) - limit
    assert over.max() <= 0, f"{what}: {over.max()} over, largest {np.abs(ref).max()}"


def _oracle_args(x):
    return [x[n] for n in ("q", "k", "v", "i", "f")]


SHAPES = [
    # B, NH, S, DK, DV, kind, state
    (1, 1, 1, 64, 64, "bf16", False),
    (1, 1, 1, 64, 64, "f32", True),
    (2, 3, 31, 64, 64, "f32", True),
    (1, 2, 32, 128, 128, "f32", True),
    (1, 2, 33, 256, 192, "f32", False),
    (2, 1, 63, 64, 192, "bf16", True),
    (1, 3, 64, 128, 128, "bf16", False),
    (3, 1, 65, 128, 64, "bf16", True),
    (1, 2, 130, 256, 512, "bf16", True),
    (2, 2, 257, 256, 128, "bf16", False),
    (1, 5, 333, 64, 448, "bf16", True),
    (1, 1, 200, 128, 320, "f32", True),
]


@pytest.mark.parametrize("B,NH,S,DK,DV,kind,state", SHAPES)
def test_forward(mt, B, NH, S, DK, DV, kind, state):
    x = _draw(1 + S, B, NH, S, DK, DV, kind, state)
    args, C0 = _gpu(x, kind)
    Hr, Cr = delta_fw(*_oracle_args(x), x["C0"])
    for h_dtype in (torch.float32, torch.bfloat16):
        H, C = mt.mlstm_delta_fw(*args, C0, h_dtype=h_dtype)
        assert H.dtype == h_dtype and C.dtype == torch.float32
        _close(H, Hr, F32, "H")
        _close(C, Cr, F32, "C")


@pytest.mark.parametrize("B,NH,S,DK,DV,kind,state", SHAPES)
def test_backward(mt, B, NH, S, DK, DV, kind, state):
    x = _draw(2 + S, B, NH, S, DK, DV, kind, state)
    args, C0 = _gpu(x, kind)
    with_dC = S % 2 == 1
    r = delta_grad(*_oracle_args(x), x["dH"], x["C0"], x["dC"] if with_dC else None)
    g = mt.mlstm_delta_bw(*args, _dev(x["dH"], _dtype(kind)), C0, _dev(x["dC"], torch.float32) if with_dC else None,
                          state_grads=True)
    for n in ("dQ", "dK", "dV", "d_i", "d_f", "dC0"):
        assert g[n].dtype == (_dtype(kind) if n in ("dQ", "dK", "dV") else torch.float32)
        rel = GATE if n == "d_f" else DK_BF16 if n == "dK" and kind == "bf16" else F32
        _close(g[n], r[n], rel, n)


@pytest.mark.parametrize("kind,hkind", [("bf16", "f32"), ("f32", "bf16")])
def test_backward_with_the_other_type_of_H(mt, kind, hkind):
    x = _draw(5, 1, 2, 97, 128, 128, kind, True, hkind)
    args, C0 = _gpu(x, kind)
    r = delta_grad(*_oracle_args(x), x["dH"], x["C0"])
    g = mt.mlstm_delta_bw(*args, _dev(x["dH"], _dtype(hkind)), C0, state_grads=True)
    for n in ("dQ", "dK", "dV", "d_i", "d_f", "dC0"):
        _close(g[n], r[n], GATE if n == "d_f" else DK_BF16 if n == "dK" and kind == "bf16" else F32, n)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gates_at_their_limits(mt, kind):
    """A forget gate at -inf clears the state (at a chunk's start, inside, twice
    in a row, at its end), +inf keeps it; an input gate at -inf writes nothing."""
    x = _draw(7, 1, 2, 200, 64, 64, kind)
    x["f"][..., [0, 17, 18, 63, 64, 127, 150]] = -np.inf
    x["f"][..., [5, 65, 130]] = np.inf
    x["i"][..., [3, 64, 100]] = -np.inf
    x["i"][..., [4, 65, 101]] = np.inf
    x["f"][:, 1, 160:] = -300.0
    x["i"][:, 1, 170:180] = -120.0
    args, C0 = _gpu(x, kind)
    Hr, Cr = delta_fw(*_oracle_args(x), x["C0"])
    H, C = mt.mlstm_delta_fw(*args, C0)
    _close(H, Hr, F32, "H")
    _close(C, Cr, F32, "C")
    r = delta_grad(*_oracle_args(x), x["dH"], x["C0"], x["dC"])
    g = mt.mlstm_delta_bw(*args, _dev(x["dH"], _dtype(kind)), C0, _dev(x["dC"], torch.float32), state_grads=True)
    for n in ("dQ", "dK", "dV", "d_i", "d_f", "dC0"):
        _close(g[n], r[n], GATE if n == "d_f" else DK_BF16 if n == "dK" and kind == "bf16" else F32, n)
    assert (g["d_f"][..., [0, 17, 18, 63, 64, 127, 150]] == 0).all()
    assert (g["d_i"][..., [3, 64, 100, 4, 65, 101]] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_one_key_written_again_and_again(mt, kind):
    """b = a = 1 and a single key: the inverse within a chunk is all ones on one
    subdiagonal, and the memory returns the last value.  Nothing decays, so the
    roundings of all chunks add up: sqrt of the chunk count."""
    x = _draw(11, 1, 2, 150, 64, 64, kind, False)
    x["k"][:] = 0.0
    x["k"][..., 5] = 1.0
    x["i"][:], x["f"][:] = np.inf, np.inf
    args, _ = _gpu(x, kind)
    H, C = mt.mlstm_delta_fw(*args)
    Hr, Cr = delta_fw(*_oracle_args(x))
    _close(H, Hr, F32, "H", 3)
    _close(C, Cr, F32, "C", 3)
    _close(C[:, :, 5], x["v"][:, :, -1].astype(np.float64), F32, "last value", 3)


def test_no_tokens(mt):
    for kind in ("bf16", "f32"):
        x = _draw(3, 2, 2, 0, 64, 64, kind)
        args, C0 = _gpu(x, kind)
        H, C = mt.mlstm_delta_fw(*args, C0)
        assert H.shape == (2, 2, 0, 64) and torch.equal(C, C0)
        assert torch.equal(mt.mlstm_delta_fw(*args)[1], torch.zeros_like(C))
        dC = _dev(x["dC"], torch.float32)
        dH = _dev(x["dH"], _dtype(kind))
        assert torch.equal(mt.mlstm_delta_bw(*args, dH, C0, dC, state_grads=True)["dC0"], dC)
        assert (mt.mlstm_delta_bw(*args, dH, C0, state_grads=True)["dC0"] == 0).all()


@pytest.mark.parametrize("B,NH,DK,DV,kind,state", [(1, 1, 64, 64, "f32", True), (2, 3, 128, 192, "bf16", True),
                                                   (3, 1, 256, 512, "bf16", False), (1, 7, 64, 128, "f32", False)])
def test_step(mt, B, NH, DK, DV, kind, state):
    x = _draw(21, B, NH, 1, DK, DV, kind, state)
    args, C0 = _gpu(x, kind)
    Hr, Cr = delta_fw(*_oracle_args(x), x["C0"])
    one = [a[:, :, 0].contiguous() for a in args]
    for h_dtype in (torch.float32, torch.bfloat16):
        h, C = mt.mlstm_delta_step(*one, C0, h_dtype=h_dtype)
        _close(h, Hr[:, :, 0], F32, "h")
        _close(C, Cr, F32, "C")
    if state:  # in place
        h2, C2 = mt.mlstm_delta_step(*one, C0, C_out=C0)
        assert C2 is C0 and torch.equal(C0, C) and torch.equal(h2, mt.mlstm_delta_step(*one, _dev(x["C0"], torch.float32))[0])


def test_prompt_then_tokens_then_norm(mt):
    """A prompt, tokens one by one on its state, the norm behind each: the run
    equals the same tokens in one pass (oracle)."""
    x = _draw(31, 2, 2, 80, 128, 192, "bf16", False)
    args, _ = _gpu(x, "bf16")
    rng = np.random.default_rng(5)
    w, b = rng.standard_normal((2, 192)).astype(np.float32), rng.standard_normal((2, 192)).astype(np.float32)
    wd, bd = _dev(w, torch.float32), _dev(b, torch.float32)
    Hr, Cr = delta_fw(*_oracle_args(x))
    yr = head_norm_fw(Hr, w, b)
    H, C = mt.mlstm_delta_fw(*[a[:, :, :70].contiguous() for a in args])
    ys = [mt.head_norm_fw(H, wd, bd)]
    for t in range(70, 80):
        h, C = mt.mlstm_delta_step(*[a[:, :, t].contiguous() for a in args], C, C_out=C)
        ys.append(mt.head_norm_fw(h[:, :, None], wd, bd))
    # the norm divides by the row's spread, about a fifth of the largest H
    _close(torch.cat(ys, 1), yr, F32, "y", 5)
    _close(C, Cr, F32, "C")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_training_run_through_autograd(mt, kind):
    """mlstm_delta with the head norm and the final state, gradients for every
    leaf from one backward pass."""
    x = _draw(41, 2, 3, 100, 64, 128, kind)
    args, C0 = _gpu(x, kind)
    rng = np.random.default_rng(6)
    w, b = 1.0 + 0.2 * rng.standard_normal((3, 128)).astype(np.float32), rng.standard_normal((3, 128)).astype(np.float32)
    leaves = [a.requires_grad_(True) for a in args + [C0, _dev(w, torch.float32), _dev(b, torch.float32)]]
    q, k, v, i, f, C0, wd, bd = leaves
    y, C = mt.mlstm_delta(q, k, v, i, f, C0, return_final_state=True, norm_weight=wd, norm_bias=bd)
    assert y.shape == (2, 100, 3, 128) and y.dtype == _dtype(kind)
    dy = rng.standard_normal(y.shape).astype(np.float32)
    if kind == "bf16":
        dy = round_to_bf16(dy)[0]
    torch.autograd.backward([y, C], [_dev(dy, _dtype(kind)), _dev(x["dC"], torch.float32)])
    Hr, Cr = delta_fw(*_oracle_args(x), x["C0"])
    dx, dw, db = head_norm_grad(Hr, dy, w)
    r = delta_grad(*_oracle_args(x), dx, x["C0"], x["dC"])
    # the gradient of H, float32, is off by the norm's own F32 and reaches
    # everything behind it linearly
    for leaf, n in zip(leaves, ("dQ", "dK", "dV", "d_i", "d_f", "dC0")):
        rel = GATE if n == "d_f" else DK_BF16 if n == "dK" and kind == "bf16" else F32
        _close(leaf.grad, r[n], rel, n, 5)
    _close(wd.grad, dw, F32, "dw", 5)
    _close(bd.grad, db, F32, "db")


def test_gradients_only_through_the_state(mt):
    x = _draw(43, 1, 2, 70, 64, 64, "f32")
    args, C0 = _gpu(x, "f32")
    leaves = [a.requires_grad_(True) for a in args + [C0]]
    _, C = mt.mlstm_delta(*leaves, return_final_state=True)
    C.backward(_dev(x["dC"], torch.float32))
    r = delta_grad(*_oracle_args(x), np.zeros_like(x["dH"]), x["C0"], x["dC"])
    for leaf, n in zip(leaves, ("dQ", "dK", "dV", "d_i", "d_f", "dC0")):
        _close(leaf.grad, r[n], GATE if n == "d_f" else F32, n)


def test_backward_against_differences(mt):
    """The directional derivative of sum(w H) from two forward passes on float32
    inputs.  Each pass is off by F32 of |H| in every value, independently over N
    values: sqrt(2 N) F32 max|H| / (2 h); the third derivative adds h^2 times
    the derivative's own size."""
    x = _draw(47, 1, 1, 70, 64, 64, "f32")
    args, C0 = _gpu(x, "f32")
    w = _dev(x["dH"], torch.float32)
    g = mt.mlstm_delta_bw(*args, w, C0, state_grads=True)
    h = 0.02
    for j, n in enumerate(("dQ", "dK", "dV", "d_i", "d_f")):
        d = torch.randn(args[j].shape, generator=torch.Generator().manual_seed(j)).cuda()
        d /= d.norm()
        out = []
        for sign in (1, -1):
            moved = list(args)
            moved[j] = args[j] + sign * h * d
            out.append((w.double() * mt.mlstm_delta_fw(*moved, C0)[0].double()).sum())
        diff, want = float(out[0] - out[1]) / (2 * h), float((g[n].double() * d.double()).sum())
        size = float(g[n].double().norm())
        H = mt.mlstm_delta_fw(*args, C0)[0]
        tol = np.sqrt(2 * H.numel()) * F32 * float(H.abs().max()) / (2 * h) + 4 * h * h * size
        assert abs(diff - want) <= tol, (n, diff, want, tol)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_equal_bits_and_rows_behind(mt, kind):
    """Two calls give equal bits; nothing is written behind H's last row, and
    the inputs stay as they are; a workspace full of NaN changes nothing."""
    x = _draw(51, 2, 2, 77, 64, 128, kind)
    args, C0 = _gpu(x, kind)
    keep = [a.clone() for a in args]
    H, C = mt.mlstm_delta_fw(*args, C0)
    desc = mt.make_delta_desc(2, 2, 77, 64, 128, qkv_dtype=mt.MLSTM_BF16 if kind == "bf16" else mt.MLSTM_F32)
    big = torch.full((H.numel() + 4096,), 7.0, device="cuda")
    out = big[:H.numel()].view(H.shape)
    ws = torch.full((mt.delta_fw_workspace_bytes(desc),), 255, dtype=torch.uint8, device="cuda")
    H2, C2 = mt.mlstm_delta_fw(*args, C0, out=out, workspace=ws)
    assert torch.equal(H, H2) and torch.equal(C, C2) and (big[H.numel():] == 7.0).all()
    dH = _dev(x["dH"], torch.float32)
    ws = torch.full((mt.delta_bw_workspace_bytes(desc),), 255, dtype=torch.uint8, device="cuda")
    g, g2 = mt.mlstm_delta_bw(*args, dH, C0, state_grads=True), mt.mlstm_delta_bw(*args, dH, C0, state_grads=True, workspace=ws)
    assert all(torch.equal(g[n], g2[n]) for n in g)
    assert all(torch.equal(a, b) for a, b in zip(args, keep))


def test_on_another_stream(mt):
    x = _draw(53, 1, 2, 130, 128, 128, "bf16")
    args, C0 = _gpu(x, "bf16")
    dH = _dev(x["dH"], torch.float32)
    H, C = mt.mlstm_delta_fw(*args, C0)
    g = mt.mlstm_delta_bw(*args, dH, C0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        H2, C2 = mt.mlstm_delta_fw(*args, C0)
        g2 = mt.mlstm_delta_bw(*args, dH, C0)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(H, H2) and torch.equal(C, C2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_captured_and_replayed(mt):
    """Forward, backward, a step and the norm in one graph, replayed between
    eager calls with new inputs each time."""
    x = _draw(57, 1, 2, 100, 64, 128, "bf16")
    args, C0 = _gpu(x, "bf16")
    dH = _dev(x["dH"], torch.float32)
    w = torch.rand(2, 128, device="cuda") + 0.5
    one = [a[:, :, 0].contiguous() for a in args]

    def work():
        H, C = mt.mlstm_delta_fw(*args, C0)
        y = mt.head_norm_fw(H, w)
        dx, dw, db = mt.head_norm_bw(H, dH.transpose(1, 2).contiguous(), w)
        g = mt.mlstm_delta_bw(*args, dx, C0, state_grads=True)
        h, C1 = mt.mlstm_delta_step(*one, C)
        return [H, C, y, dx, dw, db, h, C1] + [g[n] for n in sorted(g)]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for seed in range(3):
        y = _draw(60 + seed, 1, 2, 100, 64, 128, "bf16")
        fresh, C1 = _gpu(y, "bf16")
        for a, b in zip(args, fresh):
            a.copy_(b)
        C0.copy_(C1)
        dH.copy_(_dev(y["dH"], torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, work()):
            assert torch.equal(a, b)


def test_more_columns_a_workgroup(mt):
    """Enough heads for the walk's four- and eight-wave workgroups."""
    for B, NH, DV in ((16, 16, 64), (8, 16, 256)):
        x = _draw(71, B, NH, 70, 64, DV, "bf16")
        args, C0 = _gpu(x, "bf16")
        H, C = mt.mlstm_delta_fw(*args, C0)
        Hr, Cr = delta_fw(*_oracle_args(x), x["C0"])
        _close(H, Hr, F32, "H")
        _close(C, Cr, F32, "C")
        g = mt.mlstm_delta_bw(*args, _dev(x["dH"], torch.bfloat16), C0, state_grads=True)
        r = delta_grad(*_oracle_args(x), x["dH"], x["C0"])
        for n in ("dQ", "dK", "dV", "d_i", "d_f", "dC0"):
            _close(g[n], r[n], GATE if n == "d_f" else DK_BF16 if n == "dK" else F32, n)


def test_two_streams_at_once(mt):
    """Calls on two streams without a wait between them, each with its own
    inputs: the bits of one after the other."""
    sets = [_gpu(_draw(81 + j, 2, 2, 300, 128, 128, "bf16"), "bf16") for j in range(2)]
    dH = [_dev(_draw(83 + j, 2, 2, 300, 128, 128, "bf16")["dH"], torch.bfloat16) for j in range(2)]

    def work(j):
        args, C0 = sets[j]
        H, C = mt.mlstm_delta_fw(*args, C0)
        g = mt.mlstm_delta_bw(*args, dH[j], C0, state_grads=True)
        return [H, C, mt.head_norm_fw(H)] + [g[n] for n in sorted(g)]

    want = [work(j) for j in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((j, work(j)))
    torch.cuda.synchronize()
    for j, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[j]))


def test_two_graphs_that_share_a_workspace(mt):
    """Replayed one after the other, in any order, with eager calls on the same
    workspace between them."""
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    graphs = []
    for j, (S, DK) in enumerate(((100, 64), (150, 128))):
        x = _draw(91 + j, 1, 2, S, DK, 64, "bf16")
        args, C0 = _gpu(x, "bf16")
        dH = _dev(x["dH"], torch.bfloat16)

        def work(args=args, C0=C0, dH=dH):
            H, C = mt.mlstm_delta_fw(*args, C0, workspace=ws)
            g = mt.mlstm_delta_bw(*args, dH, C0, workspace=ws)
            return [H, C] + [g[n] for n in sorted(g)]

        want = [o.clone() for o in work()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work()
        graphs.append((graph, out, want, work))
    for j in (0, 1, 1, 0, 1, 0):
        graph, out, want, _ = graphs[j]
        for o in out:
            o.zero_()
        graph.replay()
        eager = graphs[1 - j][3]()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, graphs[1 - j][2]))


@pytest.mark.parametrize("DV,B", [(64, 1), (512, 32)])
def test_a_nan_leaves_other_heads_and_earlier_chunks(mt, DV, B):
    """Both forms of the walk (few columns, many)."""
    x = _draw(95, B, 2, 200, 64, DV, "bf16")
    args, C0 = _gpu(x, "bf16")
    H, C = mt.mlstm_delta_fw(*args, C0)
    args[1][0, 0, 100, 5] = float("nan")
    H2, C2 = mt.mlstm_delta_fw(*args, C0)
    assert H2[0, 0, 100:].isnan().any() and C2[0, 0].isnan().any()
    assert torch.equal(H2[0, 0, :64], H[0, 0, :64])
    assert torch.equal(H2[0, 1], H[0, 1]) and torch.equal(H2[1:], H[1:]) and torch.equal(C2[0, 1], C[0, 1])


def test_padding_of_zeros(mt):
    """Rows of zeros with i = -inf behind a sequence, f anything: the state
    decays by the forget gates only, the rows before are as without them, and
    their gradients too."""
    x = _draw(97, 2, 2, 90, 64, 128, "bf16")
    args, C0 = _gpu(x, "bf16")
    dH = _dev(x["dH"], torch.bfloat16)
    pad = [torch.cat([a, torch.zeros_like(a[:, :, :50])], 2) for a in args]
    pad[3][:, :, 90:] = float("-inf")
    pad[4][:, :, 90:] = float("inf")
    H, C = mt.mlstm_delta_fw(*args, C0)
    H2, C2 = mt.mlstm_delta_fw(*pad, C0)
    Hr, Cr = delta_fw(*_oracle_args(x), x["C0"])
    _close(H2[:, :, :90], Hr, F32, "H")
    _close(C2, Cr, F32, "C")
    assert (H2[:, :, 90:] == 0).all()
    dHp = torch.cat([dH, torch.ones_like(dH[:, :, :50])], 2)
    g = mt.mlstm_delta_bw(*pad, dHp, C0, state_grads=True)
    r = delta_grad(*_oracle_args(x), x["dH"], x["C0"])
    for n in ("dQ", "dK", "dV", "d_i", "d_f", "dC0"):
        rel = GATE if n == "d_f" else DK_BF16 if n == "dK" else F32
        _close(g[n] if n == "dC0" else g[n][:, :, :90], r[n], rel, n)
    assert (g["dV"][:, :, 90:] == 0).all() and (g["d_i"][:, :, 90:] == 0).all()


def test_one_tensor_for_queries_and_keys(mt):
    x = _draw(99, 1, 2, 70, 64, 64, "f32")
    x["q"] = x["k"]
    args, C0 = _gpu(x, "f32")
    key = args[1].requires_grad_(True)
    mt.mlstm_delta(key, key, *args[2:], C0).backward(_dev(x["dH"], torch.float32))
    r = delta_grad(*_oracle_args(x), x["dH"], x["C0"])
    _close(key.grad, r["dQ"] + r["dK"], F32, "dQ + dK", 2)


def test_a_broadcast_gradient(mt):
    x = _draw(101, 1, 2, 70, 64, 64, "bf16")
    args, C0 = _gpu(x, "bf16")
    leaves = [a.requires_grad_(True) for a in args]
    H = mt.mlstm_delta(*leaves, C0)
    H.sum().backward()
    g = mt.mlstm_delta_bw(*[a.detach() for a in args], torch.ones_like(H), C0)
    assert all(torch.equal(a.grad, g[n]) for a, n in zip(leaves, ("dQ", "dK", "dV", "d_i", "d_f")))


def test_refused_with_tensors_on_the_gpu(mt):
    x = _draw(103, 1, 2, 70, 64, 64, "bf16")
    args, C0 = _gpu(x, "bf16")
    dH = _dev(x["dH"], torch.bfloat16)
    q, k, v, i, f = args
    turned = q.transpose(2, 3).contiguous().transpose(2, 3)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for call in (lambda: mt.mlstm_delta_fw(turned, k, v, i, f), lambda: mt.mlstm_delta_fw(q, k[:, :, 1:], v, i, f),
                 lambda: mt.mlstm_delta_fw(q, k, v.cpu(), i, f), lambda: mt.mlstm_delta_fw(q, k, v, i, f, C0[:, :1]),
                 lambda: mt.mlstm_delta_fw(q, k, v, i, f, C0[:, :1].expand(1, 2, 64, 64)),
                 lambda: mt.mlstm_delta_fw(q, k, v, i, f, workspace=small),
                 lambda: mt.mlstm_delta_fw(q, k, v, i, f, workspace=small.cpu()),
                 lambda: mt.mlstm_delta_bw(q, k, v, i, f, dH[:, :, :69]),
                 lambda: mt.mlstm_delta_bw(q, k, v, i, f, dH, workspace=small),
                 lambda: mt.head_norm_fw(turned), lambda: mt.head_norm_bw(q, q),
                 lambda: mt.head_norm_fw(q, torch.ones(2, 32, device="cuda")),
                 lambda: mt.head_norm_fw(q, torch.ones(2, 64))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mt.mlstm_delta_fw(q, k.float(), v, i, f), lambda: mt.mlstm_delta_fw(q, k, v, i.bfloat16(), f),
                 lambda: mt.mlstm_delta_fw(q, k, v, i, f, h_dtype=torch.float16),
                 lambda: mt.head_norm_fw(q, torch.ones(2, 64, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises((TypeError, ValueError)):
            call()
    bad = torch.zeros(1, 1, 4, 96, device="cuda")
    with pytest.raises(mt.MlstmError):
        mt.mlstm_delta_fw(bad, bad, bad, bad[..., 0].contiguous(), bad[..., 0].contiguous())


def test_offsets_beyond_32_bits(mt):
    """Four million tokens of one head (Q, K over 2^31 bytes, the states 4.3
    GB): behind a closed forget gate on a chunk's border the rows are those of
    a short sequence, each side off by F32."""
    t0 = 1 << 22
    S = t0 + 77
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k = (torch.empty(1, 1, S, 256, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1 / 16, generator=gen)
            for _ in range(2))
    v, dH = (torch.empty(1, 1, S, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    i = torch.empty(1, 1, S, device="cuda").normal_(generator=gen)
    f = torch.full((1, 1, S), 3.0, device="cuda")
    f[0, 0, t0] = float("-inf")
    args = (q, k, v, i, f)
    tail = [a[:, :, t0:].contiguous() for a in args]
    H, C = mt.mlstm_delta_fw(*args)
    Ht, Ct = mt.mlstm_delta_fw(*tail)
    g = mt.mlstm_delta_bw(*args, dH)
    gt = mt.mlstm_delta_bw(*tail, dH[:, :, t0:].contiguous())
    for n, a, b in [("H", H[:, :, t0:], Ht), ("C", C, Ct)] + [(n, g[n][:, :, t0:], gt[n]) for n in g]:
        rel = GATE if n == "d_f" else DK_BF16 if n == "dK" else F32
        _close(a, b.double().cpu().numpy(), rel, n, 2)
    assert torch.isfinite(H).all() and all(torch.isfinite(x).all() for x in g.values())


def test_a_captured_training_pass(mt):
    """Forward, norm and gradients through autograd in one graph (no eager
    graph of the leaves is alive while it is captured), replayed with new
    inputs between eager passes."""
    x = _draw(111, 1, 3, 90, 64, 128, "bf16")
    args, C0 = _gpu(x, "bf16")
    w = (torch.rand(3, 128, device="cuda") + 0.5).requires_grad_(True)
    leaves = [a.requires_grad_(True) for a in args + [C0]] + [w]
    dy = _dev(x["dH"].transpose(0, 2, 1, 3), torch.bfloat16)

    def work():
        y, C = mt.mlstm_delta(*leaves[:6], return_final_state=True, norm_weight=w)
        return [y.detach(), C.detach()] + list(torch.autograd.grad([y, C], leaves, [dy, torch.ones_like(C)]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for seed in range(3):
        fresh, C1 = _gpu(_draw(112 + seed, 1, 3, 90, 64, 128, "bf16"), "bf16")
        with torch.no_grad():
            for a, b in zip(leaves, fresh + [C1]):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(got, work()))
