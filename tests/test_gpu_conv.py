"""Parity of the short causal convolution (mlstm_conv_fw, _bw, _step and the
autograd function) against the float64 oracle (needs an MI355X).

Tolerances, u = 2^-24: p is a sum of K + 1 terms, off by (K + 2) u of their
magnitudes; the sigmoid's argument is off by |p| times two roundings and its two
instructions by four, so y and its slope take (3 |p| + 12) u more, the slope of
terms up to 1 + |p|.  dx adds K products, dw and db the tokens in runs of at
most 512 and then the runs: 600 roundings of the sum of magnitudes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_bounds import U, close  # noqa: E402
from oracle import conv_fw, conv_grad  # noqa: E402
from oracle.mlstm_block import silu_slope  # noqa: E402
from workloads import round_to_bf16  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _dev(x, kind="f32"):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=TYPES[kind])


def _draw(seed, B, S, D, K, kind, bias=True, state=True):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s).astype(np.float32)
    io = lambda v: round_to_bf16(v)[0] if kind == "bf16" else v
    return dict(x=io(n(B, S, D)), w=n(D, K), bias=n(D) if bias else None, state=io(n(B, K - 1, D)) if state else None), \
        io(n(B, S, D)), io(n(B, K - 1, D))


def _bounds(kw, dy, ds, act):
    mag = {n: None if v is None else np.abs(v) for n, v in kw.items()}
    K = kw["w"].shape[1]
    P = conv_fw(**mag, act=False)[0]                     # sum of the magnitudes of p's terms
    p = conv_fw(**kw, act=False)[0]
    ep = (K + 2) * U * P
    y = np.abs(p) * (3 * np.abs(p) + 12) * U + 1.1 * ep if act else ep
    slope = np.abs(silu_slope(p)) if act else np.ones(p.shape)
    eslope = (1 + np.abs(p)) * (3 * np.abs(p) + 12) * U + 0.5 * ep if act else 0 * p   # |slope'| <= 1/2
    full = conv_grad(dy=np.abs(dy), dstate=np.abs(ds), slope=slope, **mag)
    err = conv_grad(dy=np.abs(dy), slope=eslope + (K + 4) * U * slope, **mag)
    b = {n: err[n] + (600 if n in ("dw", "db") else 4) * U * full[n] for n in full}
    return {**b, "y": y}


def _check(mt, kw, dy, ds, kind, act):
    g = {n: _dev(v, kind if n in ("x", "state") else "f32") for n, v in kw.items()}
    activation = "silu" if act else None
    y, s = mt.causal_conv_fw(g["x"], g["w"], g["bias"], g["state"], activation=activation)
    b = _bounds(kw, dy, ds, act)
    ry, rs = conv_fw(**kw, act=act)
    close(y, ry, b["y"], "y", kind)
    assert (s.double().cpu().numpy() == rs).all()
    r = mt.causal_conv_bw(g["x"], g["w"], _dev(dy, kind), g["bias"], g["state"], _dev(ds, kind), activation=activation, state_grads=True)
    ref = conv_grad(dy=dy, dstate=ds, act=act, **kw)
    for n in ("dx", "dw", "db", "dstate"):
        close(r[n], ref[n], b[n], n, kind if n in ("dx", "dstate") else "f32")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("B,S,D", [(1, 1, 1), (2, 2, 8), (1, 3, 13), (3, 4, 64), (2, 8, 40), (1, 9, 65), (2, 17, 520), (1, 130, 24),
                                   (1, 700, 7), (2, 1100, 16)])
def test_forward_and_backward(mt, B, S, D, K, kind):
    for act in (True, False):
        _check(mt, *_draw(B + S + D + K, B, S, D, K, kind), kind, act)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("bias,state", [(False, True), (True, False), (False, False)])
def test_without_bias_or_state(mt, bias, state, kind):
    for S in (1, 2, 50):
        _check(mt, *_draw(3 + S, 2, S, 48, 4, kind, bias, state), kind, True)


def test_many_rows(mt):
    """Runs of the backward pass longer than the shortest, and several workgroups a run."""
    _check(mt, *_draw(9, 4, 1500, 4104, 3, "bf16"), "bf16", True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,K", [(1, 1, 2), (3, 64, 4), (2, 77, 3), (64, 256, 4)])
def test_step(mt, B, D, K, kind):
    kw, _, _ = _draw(11, B, 1, D, K, kind)
    g = {n: _dev(v, kind if n in ("x", "state") else "f32") for n, v in kw.items()}
    x = g["x"][:, 0].contiguous()
    y, s = mt.causal_conv_step(x, g["w"], g["bias"], g["state"], activation="silu")
    y2, s2 = mt.causal_conv_fw(g["x"], g["w"], g["bias"], g["state"], activation="silu")
    assert torch.equal(y, y2[:, 0]) and torch.equal(s, s2)
    state = g["state"].clone()
    y3, s3 = mt.causal_conv_step(x, g["w"], g["bias"], state, activation="silu", state_out=state)
    assert s3 is state and torch.equal(y, y3) and torch.equal(s, state)
    y4, s4 = mt.causal_conv_step(x, g["w"])
    y5, s5 = mt.causal_conv_fw(g["x"], g["w"])
    assert torch.equal(y4, y5[:, 0]) and torch.equal(s4, s5)


def test_no_tokens(mt):
    kw, _, ds = _draw(13, 2, 0, 24, 4, "f32")
    g = {n: _dev(v) for n, v in kw.items()}
    y, s = mt.causal_conv_fw(g["x"], g["w"], g["bias"], g["state"])
    assert y.shape == (2, 0, 24) and torch.equal(s, g["state"])
    r = mt.causal_conv_bw(g["x"], g["w"], y, g["bias"], g["state"], _dev(ds), state_grads=True)
    assert torch.equal(r["dstate"], _dev(ds)) and (r["dw"] == 0).all() and (r["db"] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_runs_of_columns_and_odd_places(mt, kind):
    """A run of columns, 16-byte pieces or single values: the same bits."""
    kw, dy, ds = _draw(17, 2, 33, 64, 4, kind)
    g = {n: _dev(v, kind if n in ("x", "state") else "f32") for n, v in kw.items()}
    want = mt.causal_conv_fw(g["x"], g["w"], g["bias"], g["state"], activation="silu")
    wb = mt.causal_conv_bw(g["x"], g["w"], _dev(dy, kind), g["bias"], g["state"], _dev(ds, kind), activation="silu", state_grads=True)
    for at in (0, 8, 3):
        wide = torch.full((2, 40, 150), 5.0, dtype=TYPES[kind], device="cuda")
        wide[:, 2:35, at:at + 64] = g["x"]
        x = wide[:, 2:35, at:at + 64]
        got = mt.causal_conv_fw(x, g["w"], g["bias"], g["state"], activation="silu")
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        gb = mt.causal_conv_bw(x, g["w"], _dev(dy, kind), g["bias"], g["state"], _dev(ds, kind), activation="silu", state_grads=True)
        assert torch.equal(gb["dx"], wb["dx"]) and torch.equal(gb["dstate"], wb["dstate"])
        assert torch.equal(gb["dw"], wb["dw"]) and torch.equal(gb["db"], wb["db"])
    big = torch.full((want[0].numel() + 64,), 7.0, dtype=TYPES[kind], device="cuda")
    out = big[1:1 + want[0].numel()].view(want[0].shape)
    mt.causal_conv_fw(g["x"], g["w"], g["bias"], g["state"], activation="silu", out=out)
    assert torch.equal(out, want[0]) and big[0] == 7.0 and (big[1 + out.numel():] == 7.0).all()


def test_a_nan_reaches_its_taps_only(mt):
    kw, dy, _ = _draw(19, 1, 30, 16, 4, "f32")
    g = {n: _dev(v) for n, v in kw.items()}
    y, _ = mt.causal_conv_fw(g["x"], g["w"], g["bias"], g["state"], activation="silu")
    g["x"][0, 10, 5] = float("nan")
    y2, _ = mt.causal_conv_fw(g["x"], g["w"], g["bias"], g["state"], activation="silu")
    assert y2[0, 10:14, 5].isnan().all()
    y2[0, 10:14, 5] = y[0, 10:14, 5]
    assert torch.equal(y, y2)


def test_autograd(mt):
    kw, dy, ds = _draw(23, 2, 19, 24, 4, "f32")
    leaves = {n: _dev(v).requires_grad_(True) for n, v in kw.items()}
    y, s = mt.causal_conv(leaves["x"], leaves["w"], leaves["bias"], leaves["state"], activation="silu", return_final_state=True)
    # a gradient that begins at any element
    dyd = torch.cat([torch.zeros(1, device="cuda"), _dev(dy).flatten()])[1:].view(y.shape)
    grads = torch.autograd.grad([y, s], list(leaves.values()), [dyd, _dev(ds)])
    ref, b = conv_grad(dy=dy, dstate=ds, **kw), _bounds(kw, dy, ds, True)
    for n, got in zip(("dx", "dw", "db", "dstate"), grads):
        close(got, ref[n], b[n], n)
    s = mt.causal_conv(leaves["x"], leaves["w"], leaves["bias"], leaves["state"], return_final_state=True)[1]
    dx, = torch.autograd.grad(s, [leaves["x"]], _dev(ds))
    assert torch.equal(dx[:, -3:], _dev(ds)) and (dx[:, :-3] == 0).all()


def test_refusals_on_the_gpu(mt):
    kw, _, _ = _draw(29, 2, 12, 20, 4, "f32")
    g = {n: _dev(v) for n, v in kw.items()}
    for x, w, b, s in ((g["x"][0], g["w"], None, None), (g["x"], g["w"][:19], None, None), (g["x"], g["w"], g["bias"][:3], None),
                       (g["x"], g["w"], None, g["state"][:, :2]), (g["x"].transpose(1, 2).contiguous().transpose(1, 2), g["w"], None, None),
                       (g["x"], g["w"].cpu(), None, None), (g["x"], g["w"][:, 0], None, None)):
        with pytest.raises(ValueError):
            mt.causal_conv_fw(x, w, b, s)
    for x, w, s in ((g["x"].double(), g["w"], None), (g["x"], g["w"].bfloat16(), None), (g["x"], g["w"], g["state"].bfloat16())):
        with pytest.raises(TypeError):
            mt.causal_conv_fw(x, w, None, s)
    with pytest.raises(ValueError):
        mt.causal_conv_fw(g["x"], g["w"], activation="gelu")
    with pytest.raises(mt.MlstmError):
        mt.causal_conv_fw(g["x"], torch.zeros(20, 5, device="cuda"))


def test_outputs_apart_from_inputs(mt):
    """out and state_out that share memory with what other threads read."""
    store = torch.zeros(4 * 12 * 20, device="cuda")
    x, w = store[:480].view(2, 12, 20), torch.ones(20, 4, device="cuda")
    state = torch.zeros(3, 3, 20, device="cuda")
    for out in (x, store[20:500].view(2, 12, 20), store[240:720].view(2, 12, 20)):
        with pytest.raises(ValueError):
            mt.causal_conv_fw(x, w, out=out)
    out = store[480:].view(2, 12, 20)
    assert mt.causal_conv_fw(x, w, out=out)[0] is out
    with pytest.raises(ValueError):
        mt.causal_conv_step(x[:, 0], w, None, state[:2], state_out=state[1:])
    same = state[:2].view(2, 3, 20)
    assert mt.causal_conv_step(x[:, 0], w, None, state[:2], state_out=same)[1] is same
