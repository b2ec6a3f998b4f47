"""Outputs that share memory with an input, at the entry points of the short
causal convolution, the selective scan and dropout: refused before any launch, or
updated in place where that is offered.  On the CPU: addresses that nothing reads."""
import ctypes

import pytest

import xlstm_mlstm_chunkwise_amd as mt

OVERLAP, ARG = 10, 9
B, S, D, K, N = 2, 12, 20, 4, 16
FAR = 1 << 20


def _sizes(S, f32):
    io = 4 if f32 else 2
    row, col, state = B * S * D * io, B * S * N * io, 4 * B * D * N
    conv = dict(x=row, w=4 * D * K, b=4 * D, s=B * (K - 1) * D * io, y=row, so=B * (K - 1) * D * io)
    scan = dict(x=row, dt=row, A=4 * D * N, B=col, C=col, D=4 * D, z=row, bias=4 * D, h0=state, y=row, h=state)
    return conv, scan


def _apart(names):
    return {n: FAR * (j + 1) for j, n in enumerate(names)}


def _conv(entry, desc):
    return lambda p: getattr(mt.lib(), entry)(ctypes.byref(desc), *p.values(), None)


def _check(call, sizes, outs, in_place=()):
    """Every output against every input: at its place, in its last bytes, and with
    its own last bytes in the input's first."""
    for out in outs:
        for n in sizes:
            if n in outs:
                continue
            p = _apart(sizes)
            for at in (p[n], p[n] + sizes[n] - 16, p[n] - sizes[out] + 16):
                if (out, n) in in_place and at == p[n]:
                    continue
                assert call({**p, out: at // 16 * 16}) == OVERLAP, (out, n, at - p[n])


@pytest.mark.parametrize("f32", [True, False])
def test_convolution(f32):
    conv, _ = _sizes(S, f32)
    d = mt.make_conv_desc(B, S, D, K, dtype=0 if f32 else 1)
    _check(_conv("mlstm_conv_fw", d), conv, ("y", "so"))
    one, _ = _sizes(1, f32)
    d1 = mt.make_conv_desc(B, 1, D, K, dtype=0 if f32 else 1)
    _check(_conv("mlstm_conv_step", d1), one, ("y", "so"), {("so", "s")})
    back = dict(x=conv["x"], w=conv["w"], b=conv["b"], s=conv["s"], dy=conv["x"], dso=conv["s"], dx=conv["x"], ds=conv["s"], dw=conv["w"], db=conv["b"])
    need = mt.conv_bw_workspace_bytes(d)
    _check(lambda p: mt.lib().mlstm_conv_bw(ctypes.byref(d), *p.values(), 100 * FAR, need, None), back, ("dx", "ds", "dw", "db"))


@pytest.mark.parametrize("f32", [True, False])
def test_scan(f32):
    dtype = 0 if f32 else 1
    _, scan = _sizes(S, f32)
    d = mt.make_scan_desc(B, S, D, N, dtype=dtype)
    need = mt.scan_fw_workspace_bytes(d)
    _check(lambda p: mt.lib().mlstm_scan_fw(ctypes.byref(d), *p.values(), 100 * FAR, need, None), scan, ("y", "h"))
    _, one = _sizes(1, f32)
    d1 = mt.make_scan_desc(B, 1, D, N, dtype=dtype)
    _check(_conv("mlstm_scan_step", d1), one, ("y", "h"), {("h", "h0")})
    back = {k: v for k, v in scan.items() if k not in ("y", "h")}
    back.update(dy=scan["x"], dh=scan["h0"], dx=scan["x"], ddt=scan["x"], dA=scan["A"], dB=scan["B"], dC=scan["C"], dD=scan["D"], dz=scan["x"],
                db=scan["D"], dh0=scan["h0"])
    need_bw = mt.scan_bw_workspace_bytes(d)
    _check(lambda p: mt.lib().mlstm_scan_bw(ctypes.byref(d), *p.values(), 100 * FAR, need_bw, None), back,
           ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0"))


def test_dropout():
    d = mt.make_dropout_desc(1000, 0.1)
    sizes = dict(x=4000, r=4000, seed=16, y=4000)
    _check(_conv("mlstm_dropout", d), sizes, ("y",), {("y", "x"), ("y", "r")})


def test_views_reach_as_far_as_their_strides():
    """x (2, 12, 20) as columns of a (2, 12, 64) tensor: from its first value to its last."""
    d = mt.make_conv_desc(B, S, D, K, x_strides=(S * 64, 64))
    p = _apart(("x", "w", "b", "s", "y", "so"))
    last = 4 * ((S + S - 1) * 64 + D)
    assert _conv("mlstm_conv_fw", d)({**p, "y": p["x"] + last - 16}) == OVERLAP
    one = mt.make_scan_desc(B, 1, D, N, z_strides=(5000, 0))
    q = _apart(("x", "dt", "A", "B", "C", "D", "z", "bias", "h0", "y", "h"))
    assert _conv("mlstm_scan_step", one)({**q, "h": q["z"] + 4 * 5000}) == OVERLAP


def test_its_name():
    assert mt.status_str(OVERLAP) == "output shares memory with an input"
    e = mt.OverlapError(OVERLAP, "mlstm_conv_fw")
    assert isinstance(e, mt.MlstmError) and isinstance(e, ValueError) and "MLSTM_E_OVERLAP" in str(e)


@pytest.mark.gpu
def test_on_the_gpu():
    """The same through the binding, and outputs right beside an input."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    store = torch.zeros(4 * B * D * N, device="cuda")

    def at(i, *shape):
        size = 1
        for n in shape:
            size *= n
        return store[i:i + size].view(shape)

    n = B * D * N
    h, x, w = at(0, B, D, N), at(n, B, D), at(n + B * D, D, K)
    A, Bm = torch.full((D, N), -1.0, device="cuda"), torch.ones(B, N, device="cuda")
    step = lambda h_out, h=h, x=x, A=A: mt.selective_scan_step(x, x, A, Bm, Bm, h=h, h_out=h_out)
    for out, given in ((at(16, B, D, N), {}), (at(n - 16, B, D, N), {}), (at(n, B, D, N), {}), (at(n, B, D, N), dict(h=None)),
                       (at(2 * n, B, D, N), dict(A=at(2 * n + 32, D, N))), (h, dict(x=at(16, B, D)))):
        with pytest.raises(mt.OverlapError, match="shares memory"):
            step(out, **given)
    assert step(h)[1] is h and step(at(n + 80, B, D, N), x=at(n, B, D))[1].data_ptr() == store.data_ptr() + 4 * (n + 80)
    state = at(2 * n, B, K - 1, D)
    for out in (at(n + 4, B, K - 1, D), at(2 * n + 4, B, K - 1, D), at(n + B * D, B, K - 1, D)):
        with pytest.raises(ValueError):
            mt.causal_conv_step(x, w, None, state, state_out=out)
    assert mt.causal_conv_step(x, w, None, state, state_out=state)[1] is state
    rows, col = at(n, B, S, D), torch.ones(B, S, N, device="cuda")
    with pytest.raises(ValueError):
        mt.causal_conv_fw(rows, at(3 * n, D, K), out=at(3 * n - 400, B, S, D))
    assert mt.causal_conv_fw(rows, at(3 * n, D, K), out=at(3 * n - B * S * D, B, S, D))[0].shape == rows.shape
    with pytest.raises(ValueError):
        mt.selective_scan_fw(rows, rows, at(2 * n, D, N), col, col, out=at(2 * n + 4, B, S, D))
    one = torch.zeros(B * S * D + 4, device="cuda")
    with pytest.raises(ValueError):
        mt.dropout_fw(rows, 0.1, one[:4].view(torch.int64), out=one[:B * S * D].view(B, S, D))
