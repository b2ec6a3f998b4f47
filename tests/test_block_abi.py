"""Host-side checks of the short causal convolution's, the selective scan's and
dropout's entry points: descriptors, workspace sizes, refusals before any launch,
and the binding's own checks.  Nothing here launches a kernel."""
import ctypes

import pytest

import xlstm_mlstm_chunkwise_amd as mt

torch = pytest.importorskip("torch")

OK, NULLPTR, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, ALIGN, ARG = 0, 1, 2, 4, 5, 6, 8, 9


def _with(make, base, kw):
    return make(*{**base, **{k: kw[k] for k in kw if k in base}}.values(), **{k: kw[k] for k in kw if k not in base})


def _c(**kw):
    return _with(mt.make_conv_desc, dict(B=2, S=100, D=96, K=4), kw)


def _s(**kw):
    return _with(mt.make_scan_desc, dict(B=2, S=100, D=96, N=16), kw)


def _d(**kw):
    return _with(mt.make_dropout_desc, dict(n=1000, p=0.1), kw)


def test_struct_sizes():
    assert ctypes.sizeof(mt.ConvDesc) == 56 and ctypes.sizeof(mt.ScanDesc) == 120 and ctypes.sizeof(mt.DropoutDesc) == 48


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(S=0), OK), (dict(K=2), OK), (dict(K=3, dtype=1), OK), (dict(silu=0), OK), (dict(x_strides=(9600, 96)), OK),
    (dict(x_strides=(0, 1 << 24)), OK), (dict(x_strides=(3, 96)), OK),
    (dict(B=0), SHAPE), (dict(D=0), SHAPE), (dict(S=-1), SHAPE), (dict(K=1), SHAPE), (dict(K=5), SHAPE), (dict(D=1 << 22), SHAPE),
    (dict(S=1 << 30), SHAPE), (dict(B=1 << 16), SHAPE), (dict(B=1 << 14, S=1 << 18, D=1), SHAPE), (dict(B=1 << 10, S=1 << 20, D=1 << 12), SHAPE),
    (dict(B=2 ** 31 - 1, S=2 ** 30 - 1, D=2 ** 22 - 1), SHAPE), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(silu=2), ARG),
    (dict(x_strides=(-1, 0)), ARG), (dict(x_strides=(0, 95)), ARG), (dict(x_strides=(0, 1 << 25)), ARG), (dict(x_strides=(1 << 59, 96)), ARG)])
def test_conv_descriptor(kw, code):
    d = _c(**kw)
    assert mt.conv_validate(d) == code
    assert (mt.conv_bw_workspace_bytes(d) > 0) == (code == OK)
    if code:
        assert mt.lib().mlstm_conv_fw(ctypes.byref(d), *[4096] * 6, None) == code
        assert mt.lib().mlstm_conv_bw(ctypes.byref(d), *[4096] * 11, 0, None) == code
        assert mt.lib().mlstm_conv_step(ctypes.byref(d), *[4096] * 6, None) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(S=0), OK), (dict(N=32), OK), (dict(N=64, dtype=1), OK), (dict(z_strides=(19200, 192), B_strides=(800, 38)), OK),
    (dict(B=0), SHAPE), (dict(D=0), SHAPE), (dict(S=-1), SHAPE), (dict(N=0), SHAPE), (dict(N=8), SHAPE), (dict(N=48), SHAPE), (dict(N=128), SHAPE),
    (dict(D=1 << 22), SHAPE), (dict(S=1 << 30), SHAPE), (dict(B=1 << 20), SHAPE), (dict(B=1 << 12, D=1 << 14), SHAPE),
    (dict(B=1 << 10, S=1 << 20, D=1 << 12), SHAPE), (dict(B=2 ** 31 - 1, S=2 ** 30 - 1, D=2 ** 22 - 1), SHAPE), (dict(dtype=3), DTYPE),
    (dict(x_strides=(0, 95)), ARG), (dict(dt_strides=(-5, 0)), ARG), (dict(z_strides=(0, 1 << 25)), ARG), (dict(B_strides=(0, 15)), ARG),
    (dict(C_strides=(1 << 60, 0)), ARG)])
def test_scan_descriptor(kw, code):
    d = _s(**kw)
    assert mt.scan_validate(d) == code
    assert (mt.scan_fw_workspace_bytes(d) > 0) == (mt.scan_bw_workspace_bytes(d) > 0) == (code == OK and d.S > 0)
    if code:
        assert mt.lib().mlstm_scan_fw(ctypes.byref(d), *[4096] * 12, 0, None) == code
        assert mt.lib().mlstm_scan_bw(ctypes.byref(d), *[4096] * 21, 0, None) == code
        assert mt.lib().mlstm_scan_step(ctypes.byref(d), *[4096] * 11, None) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(n=0), OK), (dict(n=1 << 40), OK), (dict(p=0.0), OK), (dict(p=1 - 2.0 ** -53), OK), (dict(dtype=1), OK),
    (dict(n=-1), SHAPE), (dict(n=(1 << 40) + 1), SHAPE), (dict(p=1.0), ARG), (dict(p=-1e-9), ARG), (dict(p=float("nan")), ARG), (dict(dtype=2), DTYPE)])
def test_dropout_descriptor(kw, code):
    d = _d(**kw)
    assert mt.dropout_validate(d) == code
    if code:
        assert mt.lib().mlstm_dropout(ctypes.byref(d), *[4096] * 4, None) == code


def test_reserved_fields():
    for make, validate, n in ((_c, mt.conv_validate, 4), (_s, mt.scan_validate, 4), (_d, mt.dropout_validate, 3)):
        for i in range(n):
            d = make()
            d.reserved[i] = 1
            assert validate(d) == ARG
    d = _s()
    d.reserved0 = 1
    assert mt.scan_validate(d) == ARG


def _refusals(call, names, required, align, ws_need):
    """Every required pointer, every alignment (align: name -> bytes), the workspace."""
    good = {n: 4096 * (j + 1) for j, n in enumerate(names)}
    for n in required:
        assert call({**good, n: None}, ws_need) == NULLPTR, n
    for n in names:
        if n != "ws":
            assert call({**good, n: good[n] + align.get(n, 4) // 2}, ws_need) == ALIGN, n
    if ws_need:
        assert call({**good, "ws": None}, ws_need) == WORKSPACE
        assert call(good, ws_need - 1) == WORKSPACE
        assert call({**good, "ws": good["ws"] + 128}, ws_need) == WORKSPACE


@pytest.mark.parametrize("dtype", [0, 1])
def test_conv_refuses_before_launch(dtype):
    io = 2 if dtype else 4
    d, names = _c(dtype=dtype), ("x", "w", "b", "s", "y", "so")
    at = {n: io for n in ("x", "s", "y", "so", "dy", "dso", "dx", "ds")}
    lib = mt.lib()
    _refusals(lambda p, n: lib.mlstm_conv_fw(ctypes.byref(d), *p.values(), None), names, ("x", "w", "y"), at, 0)
    _refusals(lambda p, n: lib.mlstm_conv_bw(ctypes.byref(d), *p.values(), n, None),
              ("x", "w", "b", "s", "dy", "dso", "dx", "ds", "dw", "db", "ws"), ("x", "w", "dy", "dx"), at, mt.conv_bw_workspace_bytes(d))
    one = _c(S=1, dtype=dtype)
    _refusals(lambda p, n: lib.mlstm_conv_step(ctypes.byref(one), *p.values(), None), names, ("x", "w", "y", "so"), at, 0)
    for S in (0, 2):
        assert lib.mlstm_conv_step(ctypes.byref(_c(S=S)), *[4096] * 6, None) == SHAPE
    assert lib.mlstm_conv_fw(None, *[4096] * 6, None) == NULLPTR


@pytest.mark.parametrize("dtype", [0, 1])
def test_scan_refuses_before_launch(dtype):
    io = 2 if dtype else 4
    at = {n: io for n in ("x", "dt", "B", "C", "z", "y", "dy", "dx", "ddt", "dB", "dC", "dz")}
    at.update({n: 16 for n in ("A", "h0", "h", "dh", "dA", "dh0")})
    lib, d = mt.lib(), _s(dtype=dtype)
    ins = ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0")
    _refusals(lambda p, n: lib.mlstm_scan_fw(ctypes.byref(d), *p.values(), n, None), ins + ("y", "h", "ws"), ("x", "dt", "A", "B", "C", "y"), at,
              mt.scan_fw_workspace_bytes(d))
    names = ins + ("dy", "dh", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "db", "dh0", "ws")
    need = mt.scan_bw_workspace_bytes(d)
    call = lambda p, n: lib.mlstm_scan_bw(ctypes.byref(d), *p.values(), n, None)
    _refusals(call, names, ("x", "dt", "A", "B", "C", "dy", "dx", "ddt", "dA", "dB", "dC", "dz"), at, need)
    good = {n: 4096 * (j + 1) for j, n in enumerate(names)}
    assert call({**good, "z": None}, need) == UNSUPPORTED
    one = _s(S=1, dtype=dtype)
    _refusals(lambda p, n: lib.mlstm_scan_step(ctypes.byref(one), *p.values(), None), ins + ("y", "h"), ("x", "dt", "A", "B", "C", "y", "h"), at, 0)
    for S in (0, 2):
        assert lib.mlstm_scan_step(ctypes.byref(_s(S=S)), *[4096] * 11, None) == SHAPE
    assert lib.mlstm_scan_fw(None, *[4096] * 12, 0, None) == NULLPTR


def test_dropout_refuses_before_launch():
    d = _d()
    call = lambda p, n: mt.lib().mlstm_dropout(ctypes.byref(d), *p.values(), None)
    _refusals(call, ("x", "r", "seed", "y"), ("x", "y"), {"seed": 8}, 0)
    assert mt.lib().mlstm_dropout(None, *[4096] * 4, None) == NULLPTR
    assert mt.lib().mlstm_dropout(ctypes.byref(_d(n=0)), None, None, None, None, None) == OK


def test_the_cut_leaves_no_piece_empty():
    """Chunks and spans of every length: the workspace counts them, and more
    tokens never take less."""
    for N in (16, 32, 64):
        for B, D in ((1, 64), (3, 960), (8, 4096), (40, 70)):
            fw = [mt.scan_fw_workspace_bytes(_s(B=B, D=D, N=N, S=S)) for S in (1, 2, 16, 17, 64, 1000, 1024, 8192)]
            assert all(v >= B * ((S + 15) // 16 * 16) * 2 * N * 4 for v, S in zip(fw, (1, 2, 16, 17, 64, 1000, 1024, 8192)))
            bw = [mt.scan_bw_workspace_bytes(_s(B=B, D=D, N=N, S=S)) for S in (1, 2, 16, 17, 64, 1000, 1024, 8192)]
            assert all(b > f for b, f in zip(bw, fw)) and bw == sorted(bw)


def test_the_binding_refuses():
    x, w, A, b = torch.zeros(1, 4, 64), torch.zeros(64, 4), torch.zeros(64, 16), torch.zeros(1, 4, 16)
    for call in (lambda: mt.causal_conv_fw(x, w), lambda: mt.causal_conv_bw(x, w, x), lambda: mt.causal_conv(x, w),
                 lambda: mt.causal_conv_step(x[:, 0], w), lambda: mt.causal_conv_fw(x[0], w), lambda: mt.causal_conv_step(x, w),
                 lambda: mt.selective_scan_fw(x, x, A, b, b), lambda: mt.selective_scan_bw(x, x, A, b, b, x),
                 lambda: mt.selective_scan(x, x, A, b, b), lambda: mt.selective_scan_step(x[:, 0], x[:, 0], A, b[:, 0], b[:, 0]),
                 lambda: mt.selective_scan_fw(x[0], x, A, b, b), lambda: mt.selective_scan_step(x, x, A, b, b),
                 lambda: mt.dropout_fw(x, 0.1, 1), lambda: mt.dropout(x, 0.1, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mt.causal_conv_fw(x.double(), w)
    for seed in (2 ** 64, -2 ** 63 - 1):
        with pytest.raises(ValueError):
            mt.make_dropout_desc(1, 0.1, seed)
    assert mt.make_dropout_desc(1, 0.1, 2 ** 64 - 1).seed == -1
