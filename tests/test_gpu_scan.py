"""Parity of the selective scan (mlstm_scan_fw, _bw, _step and the autograd
function) against the float64 oracle (needs an MI355X).  Tolerances: the bounds
of block_bounds, and the rounding of bf16 outputs on top."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_bounds import close, scan_bounds  # noqa: E402
from oracle import scan_fw, scan_grad  # noqa: E402
from workloads import round_to_bf16  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IO = ("x", "dt", "Bm", "Cm", "z")
GRADS = (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("D", "dD"), ("z", "dz"), ("dt_bias", "dbias"), ("h0", "dh0"))


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _draw(seed, B, S, D, N, kind, drop=()):
    """Inputs by name (those in drop are None), dy and dh."""
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    kw = dict(x=n((B, S, D)), dt=0.7 * n((B, S, D)), A=-np.arange(1, N + 1) * np.exp(0.1 * n((D, N))), Bm=n((B, S, N)),
              Cm=n((B, S, N)), D=1 + 0.1 * n(D), z=n((B, S, D)), dt_bias=rng.uniform(-6.0, -1.0, D), h0=0.3 * n((B, D, N)),
              dy=n((B, S, D)), dh=n((B, D, N)))
    for name, v in kw.items():
        v = v.astype(np.float32)
        kw[name] = None if name in drop else round_to_bf16(v)[0] if kind == "bf16" and name in IO + ("dy",) else v
    return {k: kw[k] for k in kw if k not in ("dy", "dh")}, kw["dy"], kw["dh"]


def _dev(x, kind="f32"):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=TYPES[kind])


def _gpu(kw, kind):
    return {n: _dev(v, kind if n in IO else "f32") for n, v in kw.items()}


def _args(g):
    return [g[n] for n in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")]


def _bw(mt, g, dy, dh, **more):
    a = _args(g)
    return mt.selective_scan_bw(*a[:5], dy, *a[5:], dh, state_grads=True, **more)


def _check(mt, kw, dy, dh, kind):
    g = _gpu(kw, kind)
    y, h = mt.selective_scan_fw(*_args(g))
    b = scan_bounds(kw, dy, dh)
    ry, rh = scan_fw(**kw)
    close(y, ry, b["y"], "y", kind)
    close(h, rh, b["h"], "h")
    got, ref = _bw(mt, g, _dev(dy, kind), _dev(dh)), scan_grad(dy=dy, dh=dh, **kw)
    assert ("dz" in got) == (kw["z"] is not None)
    for name in got:
        close(got[name], ref[name], b[name], name, kind if name in ("dx", "ddt", "dB", "dC", "dz") else "f32")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,S,D,N", [
    (1, 1, 1, 16), (2, 1, 64, 32), (1, 2, 33, 64), (1, 7, 17, 16), (2, 8, 65, 16), (1, 9, 128, 32), (3, 15, 31, 16),
    (1, 16, 129, 64), (2, 17, 96, 16), (1, 31, 16, 32), (1, 32, 200, 16), (2, 33, 48, 64), (1, 63, 64, 16), (1, 64, 64, 64),
    (1, 65, 130, 32), (1, 127, 70, 16), (2, 200, 40, 16), (1, 333, 20, 64), (1, 400, 24, 32)])
def test_forward_and_backward(mt, B, S, D, N, kind):
    _check(mt, *_draw(B + S + D + N, B, S, D, N, kind), kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("drop", [("z",), ("D", "dt_bias", "h0"), ("z", "D", "dt_bias", "h0", "dh")])
def test_without_the_optional_inputs(mt, drop, kind):
    for N in (16, 64):
        _check(mt, *_draw(5, 2, 75, 50, N, kind, drop), kind)


@pytest.mark.parametrize("B,D,N", [(4, 4100, 16), (3, 2100, 64)])
def test_many_channels(mt, B, D, N):
    """Enough workgroups for one chunk and one span (no pieces side by side)."""
    desc = mt.make_scan_desc(B, 40, D, N)
    assert mt.scan_fw_workspace_bytes(desc) == B * 48 * 2 * N * 4
    _check(mt, *_draw(7, B, 40, D, N, "f32"), "f32")


def test_large_and_small_steps(mt):
    """Steps from e^-30 to 60: decays from one to zero."""
    kw, dy, dh = _draw(11, 1, 90, 64, 16, "f32")
    kw["dt"] = np.random.default_rng(1).uniform(-30, 60, kw["dt"].shape).astype(np.float32)
    _check(mt, kw, dy, dh, "f32")


@pytest.mark.parametrize("N", [16, 32, 64])
def test_padding(mt, N):
    """dt = -inf leaves the state as it is, bit by bit, in front of and behind the
    tokens and between them."""
    kw, dy, _ = _draw(13, 1, 50, 40, N, "bf16")
    keep = np.r_[3:20, 24:45]
    kw["dt"][:] = -np.inf
    kw["dt"][:, keep] = 0.5
    y, h = mt.selective_scan_fw(*_args(_gpu(kw, "bf16")))
    one = _gpu(kw, "bf16")
    state = one["h0"]
    for t in range(50):
        before = state
        yt, state = mt.selective_scan_step(*[one[n][:, t] for n in ("x", "dt")], one["A"], one["Bm"][:, t], one["Cm"][:, t], one["D"],
                                           one["z"][:, t], one["dt_bias"], state)
        if t not in keep:
            assert torch.equal(before, state)
    b = scan_bounds({n: v for n, v in kw.items()})
    assert (h - state).abs().double().cpu().numpy().max() <= 2 * b["h"].max()
    g = _bw(mt, one, _dev(dy, "bf16"), None)
    gone = np.setdiff1d(np.arange(50), keep)
    assert (g["ddt"][:, gone] == 0).all()
    ref = scan_grad(dy=dy, **kw)
    assert np.isfinite(ref["dA"]).all()
    close(g["dA"], ref["dA"], scan_bounds(kw, dy)["dA"], "dA")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,N", [(1, 1, 16), (3, 65, 16), (2, 40, 32), (5, 33, 64), (64, 128, 16)])
def test_step(mt, B, D, N, kind):
    kw, _, _ = _draw(17 + D, B, 1, D, N, kind)
    g = _gpu(kw, kind)
    ry, rh = scan_fw(**kw)
    b = scan_bounds(kw)

    def step(h, **more):
        a = [v[:, 0] if n in IO else v for n, v in g.items()]
        x, dt, A, Bm, Cm, D_, z, bias, _ = a
        return mt.selective_scan_step(x, dt, A, Bm, Cm, D_, z, bias, h, **more)

    y, h = step(g["h0"])
    close(y, ry[:, 0], b["y"][:, 0], "y", kind)
    close(h, rh, b["h"], "h")
    state = g["h0"].clone()
    y2, h2 = step(state, h_out=state)
    assert h2 is state and torch.equal(y, y2) and torch.equal(h, h2)
    none = {**kw, "h0": None}
    y3, h3 = step(None)
    close(h3, scan_fw(**none)[1], scan_bounds(none)["h"], "h")


def test_no_tokens(mt):
    kw, _, dh = _draw(19, 2, 0, 30, 16, "f32")
    g = _gpu(kw, "f32")
    y, h = mt.selective_scan_fw(*_args(g))
    assert y.shape == (2, 0, 30) and torch.equal(h, g["h0"])
    assert (mt.selective_scan_fw(*_args(g)[:8])[1] == 0).all()
    r = _bw(mt, g, y, _dev(dh))
    assert torch.equal(r["dh0"], _dev(dh)) and all((r[n] == 0).all() for n in ("dA", "dD", "dbias")) and r["dx"].shape == (2, 0, 30)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_runs_of_columns(mt, kind):
    """x, dt, z, B and C as columns of wider tensors, at odd places: the bits of
    contiguous ones; a batch whose rows lie behind each other with a gap."""
    kw, dy, dh = _draw(23, 2, 45, 70, 16, kind)
    g = _gpu(kw, kind)
    wide = torch.full((2, 45, 300), 3.0, dtype=TYPES[kind], device="cuda")
    at = {"x": 1, "dt": 73, "z": 150, "Bm": 223, "Cm": 241}
    v = dict(g)
    for n, a in at.items():
        wide[..., a:a + g[n].shape[-1]] = g[n]
        v[n] = wide[..., a:a + g[n].shape[-1]]
    tall = torch.zeros((2, 60, 70), dtype=TYPES[kind], device="cuda")
    tall[:, 5:50] = g["x"]
    for views in (v, {**g, "x": tall[:, 5:50]}):
        y, h = mt.selective_scan_fw(*_args(g))
        y2, h2 = mt.selective_scan_fw(*_args(views))
        assert torch.equal(y, y2) and torch.equal(h, h2)
        r, r2 = _bw(mt, g, _dev(dy, kind), _dev(dh)), _bw(mt, views, _dev(dy, kind), _dev(dh))
        assert all(torch.equal(r[n], r2[n]) for n in r)
    y, h = mt.selective_scan_step(v["x"][:, 3], v["dt"][:, 3], v["A"], v["Bm"][:, 3], v["Cm"][:, 3], v["D"], v["z"][:, 3], v["dt_bias"], v["h0"])
    y2, h2 = mt.selective_scan_step(*[g[n][:, 3].contiguous() for n in ("x", "dt")], g["A"], g["Bm"][:, 3].contiguous(),
                                    g["Cm"][:, 3].contiguous(), g["D"], g["z"][:, 3].contiguous(), g["dt_bias"], g["h0"])
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_continued(mt):
    """A sequence in two calls is the sequence in one."""
    kw, _, _ = _draw(29, 2, 100, 50, 16, "f32")
    g = _gpu(kw, "f32")
    y, h = mt.selective_scan_fw(*_args(g))
    first = {n: (v[:, :37].contiguous() if n in IO else v) for n, v in g.items()}
    second = {n: (v[:, 37:].contiguous() if n in IO else v) for n, v in g.items()}
    y1, h1 = mt.selective_scan_fw(*_args(first))
    y2, h2 = mt.selective_scan_fw(*_args({**second, "h0": h1}))
    b = scan_bounds(kw)
    assert (np.abs((torch.cat([y1, y2], 1) - y).double().cpu().numpy()) <= 2 * b["y"]).all()
    assert (np.abs((h2 - h).double().cpu().numpy()) <= 2 * b["h"]).all()


def test_a_nan_stays_in_its_channel(mt):
    """x, dt, z or dy that are not finite: other channels keep their bits, but
    dB and dC of tokens that it reaches; tokens before keep theirs in the
    forward pass."""
    kw, dy, dh = _draw(31, 1, 60, 70, 16, "f32")
    base = _gpu(kw, "f32")
    y, h = mt.selective_scan_fw(*_args(base))
    r = _bw(mt, base, _dev(dy), _dev(dh))
    other = torch.arange(70, device="cuda") != 37
    for name, bad in (("x", np.nan), ("dt", np.nan), ("z", np.nan), ("x", np.inf), ("dy", np.nan)):
        kw2, dy2 = {n: (v.copy() if v is not None else None) for n, v in kw.items()}, dy.copy()
        (dy2 if name == "dy" else kw2[name])[0, 21, 37] = bad
        g = _gpu(kw2, "f32")
        y2, h2 = mt.selective_scan_fw(*_args(g))
        assert torch.equal(y2[..., other], y[..., other]) and torch.equal(h2[:, other], h[:, other])
        assert torch.equal(y2[:, :21], y[:, :21])
        if name != "dy":
            assert not torch.isfinite(y2[0, 21, 37])
        r2 = _bw(mt, g, _dev(dy2), _dev(dh))
        for n in ("dx", "ddt", "dz"):
            assert torch.equal(r2[n][..., other], r[n][..., other]), (name, n)
        for n in ("dA", "dD", "dbias"):
            assert torch.equal(r2[n][other], r[n][other]), (name, n)


def test_equal_bits_and_nothing_behind(mt):
    kw, dy, dh = _draw(37, 2, 150, 100, 16, "bf16")
    g = _gpu(kw, "bf16")
    keep = [None if v is None else v.clone() for v in g.values()]
    y, h = mt.selective_scan_fw(*_args(g))
    desc = mt.make_scan_desc(2, 150, 100, 16, dtype=mt.MLSTM_BF16)
    big = torch.full((y.numel() + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((mt.scan_fw_workspace_bytes(desc),), 255, dtype=torch.uint8, device="cuda")
    y2, h2 = mt.selective_scan_fw(*_args(g), out=big[:y.numel()].view(y.shape), workspace=ws)
    assert torch.equal(y, y2) and torch.equal(h, h2) and (big[y.numel():] == 7.0).all()
    ws = torch.full((mt.scan_bw_workspace_bytes(desc),), 255, dtype=torch.uint8, device="cuda")
    r, r2 = _bw(mt, g, _dev(dy, "bf16"), _dev(dh)), _bw(mt, g, _dev(dy, "bf16"), _dev(dh), workspace=ws)
    assert all(torch.equal(r[n], r2[n]) for n in r)
    assert all(a is None or torch.equal(a, b) for a, b in zip(g.values(), keep))
    assert mt.selective_scan_fw(*_args(g), return_final_state=False)[1] is None


@pytest.mark.parametrize("S,N", [(21, 16), (40, 32)])
def test_autograd(mt, S, N):
    """Gradients through y and the final state; a shared B and C; leaves that are
    views; nothing for what needs nothing."""
    kw, dy, dh = _draw(41, 2, S, 30, N, "f32")
    g = _gpu(kw, "f32")
    leaves = {n: v.requires_grad_(True) for n, v in g.items()}
    y, h = mt.selective_scan(*_args(leaves), return_final_state=True)
    grads = torch.autograd.grad([y, h], list(leaves.values()), [_dev(dy), _dev(dh)])
    ref, b = scan_grad(dy=dy, dh=dh, **kw), scan_bounds(kw, dy, dh)
    for (n, k), got in zip(((n, dict(GRADS)[n]) for n in leaves), grads):
        close(got, ref[k], b[k], k)
    h = mt.selective_scan(*_args(leaves), return_final_state=True)[1]
    only = torch.autograd.grad(h, [leaves["x"], leaves["A"]], _dev(dh))
    ref, b = scan_grad(dy=0 * dy, dh=dh, **kw), scan_bounds(kw, 0 * dy, dh)
    close(only[0], ref["dx"], b["dx"], "dx")
    close(only[1], ref["dA"], b["dA"], "dA")
    # one tensor as B and C: its gradient is the sum
    shared = leaves["Bm"]
    y = mt.selective_scan(leaves["x"], leaves["dt"], leaves["A"], shared, shared)
    got, = torch.autograd.grad(y, [shared], _dev(dy))
    one = {"x": kw["x"], "dt": kw["dt"], "A": kw["A"], "Bm": kw["Bm"], "Cm": kw["Bm"]}
    ref, b = scan_grad(dy=dy, **one), scan_bounds(one, dy)
    close(got, ref["dB"] + ref["dC"], b["dB"] + b["dC"] + 2.0 ** -24 * np.abs(ref["dB"] + ref["dC"]), "dB + dC")


def test_a_saved_input_that_changed_is_refused(mt):
    kw, dy, _ = _draw(43, 1, 10, 20, 16, "f32")
    g = _gpu(kw, "f32")
    x = g["x"].requires_grad_(True)
    y = mt.selective_scan(*_args(g))
    g["A"].mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        torch.autograd.grad(y, [x], _dev(dy))


def test_refusals_on_the_gpu(mt):
    kw, dy, _ = _draw(47, 2, 12, 20, 16, "f32")
    g = _gpu(kw, "f32")

    def call(**over):
        return mt.selective_scan_fw(*_args({**g, **over}))

    for over in (dict(dt=g["dt"][:, :11]), dict(Bm=g["Cm"][..., :15]), dict(A=g["A"][:19]), dict(h0=g["h0"][:1]),
                 dict(z=g["z"].expand(2, 12, 20).transpose(1, 2).contiguous().transpose(1, 2)), dict(D=g["D"].cpu()),
                 dict(x=g["x"][:, :1].expand(2, 12, 20)), dict(Bm=g["Bm"].cpu()), dict(A=g["A"][0])):
        with pytest.raises(ValueError):
            call(**over)
    for over in (dict(dt=g["dt"].bfloat16()), dict(A=g["A"].double()), dict(h0=g["h0"].bfloat16())):
        with pytest.raises(TypeError):
            call(**over)
    with pytest.raises(mt.MlstmError):
        call(A=g["A"][:, :8].contiguous(), Bm=g["Bm"][..., :8], Cm=g["Cm"][..., :8], h0=g["h0"][..., :8].contiguous())
    with pytest.raises(ValueError):
        mt.selective_scan_fw(*_args(g), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mt.selective_scan_bw(*_args(g)[:5], _dev(dy)[:, :5])


def test_outputs_apart_from_inputs(mt):
    """out and h_out that share memory with what other threads read."""
    kw, _, _ = _draw(53, 2, 12, 20, 16, "f32")
    g = _gpu(kw, "f32")
    for out in (g["x"], g["dt"], g["z"]):
        with pytest.raises(ValueError):
            mt.selective_scan_fw(*_args(g), out=out)
    out = torch.empty_like(g["x"])
    assert mt.selective_scan_fw(*_args(g), out=out)[0] is out
    h = torch.zeros(3, 20, 16, device="cuda")
    x, dt, A, B, C = (v if v is g["A"] else v[:, 0] for v in _args(g)[:5])
    with pytest.raises(ValueError):
        mt.selective_scan_step(x, dt, A, B, C, h=h[:2], h_out=h[1:])
    same = h[:2].view(2, 20, 16)
    assert mt.selective_scan_step(x, dt, A, B, C, h=h[:2], h_out=same)[1] is same
