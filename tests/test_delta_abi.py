"""Host-side checks of the gated delta rule's and the head norm's entry points:
descriptors, workspace sizes, refusals before any launch, and the binding's own
checks.  Nothing here launches a kernel."""
import ctypes

import pytest

import xlstm_mlstm_chunkwise_amd as mt

torch = pytest.importorskip("torch")

OK, NULLPTR, SHAPE, DTYPE, WORKSPACE, ALIGN, ARG = 0, 1, 2, 4, 6, 8, 9


def _d(**kw):
    base = dict(B=2, NH=3, S=100, DHQK=128, DHV=192)
    base.update({k: kw.pop(k) for k in list(kw) if k in base})
    return mt.make_delta_desc(*base.values(), **kw)


def _n(**kw):
    base = dict(B=2, NH=3, S=100, D=192)
    base.update({k: kw.pop(k) for k in list(kw) if k in base})
    return mt.make_head_norm_desc(*base.values(), **kw)


def test_struct_sizes():
    assert ctypes.sizeof(mt.DeltaDesc) == 12 * 4 and ctypes.sizeof(mt.HeadNormDesc) == 10 * 4


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(S=0), OK), (dict(S=1), OK), (dict(qkv_dtype=0), OK), (dict(h_dtype=1), OK), (dict(qk_scale=0.5), OK),
    (dict(B=0), SHAPE), (dict(NH=-1), SHAPE), (dict(S=-1), SHAPE), (dict(S=(1 << 30) + 1, B=1, NH=1), SHAPE),
    (dict(DHQK=96), SHAPE), (dict(DHQK=192), SHAPE), (dict(DHQK=512), SHAPE), (dict(DHQK=0), SHAPE),
    (dict(DHV=0), SHAPE), (dict(DHV=96), SHAPE), (dict(DHV=576), SHAPE),
    (dict(B=1 << 16, NH=1 << 16), SHAPE), (dict(B=1 << 14, NH=1 << 9), SHAPE), (dict(B=1 << 20, NH=1, DHV=512), SHAPE),
    (dict(qkv_dtype=2), DTYPE), (dict(h_dtype=-1), DTYPE),
    (dict(qk_scale=float("inf")), ARG), (dict(qk_scale=float("nan")), ARG)])
def test_delta_descriptor(kw, code):
    d = _d(**kw)
    assert mt.delta_validate(d) == code
    if code:
        assert mt.delta_fw_workspace_bytes(d) == 0 == mt.delta_bw_workspace_bytes(d)
        assert mt.lib().mlstm_delta_fw(ctypes.byref(d), *[4096] * 9, 0, None) == code
        assert mt.lib().mlstm_delta_bw(ctypes.byref(d), *[4096] * 15, 0, None) == code
        assert mt.lib().mlstm_delta_step(ctypes.byref(d), *[4096] * 8, None) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(S=0), OK), (dict(x_dtype=1, y_dtype=0), OK), (dict(eps=0.0), OK),
    (dict(B=0), SHAPE), (dict(NH=0), SHAPE), (dict(S=-1), SHAPE), (dict(D=32), SHAPE), (dict(D=0), SHAPE), (dict(D=100), SHAPE),
    (dict(D=576), SHAPE), (dict(B=1 << 10, NH=1 << 10, S=1 << 10), SHAPE), (dict(B=1 << 30, NH=1 << 30, S=1 << 30), SHAPE),
    (dict(NH=1 << 22, S=0), SHAPE), (dict(x_dtype=5), DTYPE), (dict(y_dtype=-1), DTYPE),
    (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG)])
def test_norm_descriptor(kw, code):
    d = _n(**kw)
    assert mt.head_norm_validate(d) == code
    assert (mt.head_norm_bw_workspace_bytes(d) > 0) == (code == OK)
    if code:
        assert mt.lib().mlstm_head_norm_fw(ctypes.byref(d), *[4096] * 4, None) == code
        assert mt.lib().mlstm_head_norm_bw(ctypes.byref(d), *[4096] * 7, 0, None) == code


def test_reserved_fields():
    for i in range(4):
        d = _d()
        d.reserved[i] = 1
        assert mt.delta_validate(d) == ARG
    for i in range(3):
        d = _n()
        d.reserved[i] = 1
        assert mt.head_norm_validate(d) == ARG


def _refusals(call, names, required, aligned16, ws_need):
    """Every required pointer, every alignment, the workspace."""
    good = {n: 4096 * (j + 1) for j, n in enumerate(names)}
    for n in required:
        assert call({**good, n: None}, ws_need) == NULLPTR, n
    for n in names:
        if n != "ws":
            assert call({**good, n: good[n] + (8 if n in aligned16 else 2)}, ws_need) == ALIGN, n
    if ws_need:
        assert call({**good, "ws": None}, ws_need) == WORKSPACE
        assert call(good, ws_need - 1) == WORKSPACE
        assert call({**good, "ws": good["ws"] + 128}, ws_need) == WORKSPACE


def test_delta_fw_refuses_before_launch():
    d, names = _d(), ("q", "k", "v", "i", "f", "C0", "H", "C", "ws")
    _refusals(lambda p, n: mt.lib().mlstm_delta_fw(ctypes.byref(d), *p.values(), n, None), names,
              ("q", "k", "v", "i", "f", "H"), ("q", "k", "v", "H"), mt.delta_fw_workspace_bytes(d))
    assert mt.lib().mlstm_delta_fw(None, *[4096] * 9, 0, None) == NULLPTR


def test_delta_bw_refuses_before_launch():
    d, names = _d(), ("q", "k", "v", "i", "f", "C0", "dH", "dC", "dq", "dk", "dv", "di", "df", "dC0", "ws")
    _refusals(lambda p, n: mt.lib().mlstm_delta_bw(ctypes.byref(d), *p.values(), n, None), names,
              ("q", "k", "v", "i", "f", "dH", "dq", "dk", "dv", "di", "df"), ("q", "k", "v", "dH", "dq", "dk", "dv"),
              mt.delta_bw_workspace_bytes(d))
    assert mt.lib().mlstm_delta_bw(None, *[4096] * 15, 0, None) == NULLPTR


def test_delta_step_refuses_before_launch():
    d, names = _d(S=1), ("q", "k", "v", "i", "f", "C", "h", "Co")
    _refusals(lambda p, n: mt.lib().mlstm_delta_step(ctypes.byref(d), *p.values(), None), names,
              ("q", "k", "v", "i", "f", "h", "Co"), ("q", "k", "v", "C", "h", "Co"), 0)
    for S in (0, 2):
        assert mt.lib().mlstm_delta_step(ctypes.byref(_d(S=S)), *[4096] * 8, None) == SHAPE


def test_head_norm_refuses_before_launch():
    d = _n()
    _refusals(lambda p, n: mt.lib().mlstm_head_norm_fw(ctypes.byref(d), *p.values(), None), ("x", "w", "b", "y"), ("x", "y"),
              ("x", "w", "b", "y"), 0)
    _refusals(lambda p, n: mt.lib().mlstm_head_norm_bw(ctypes.byref(d), *p.values(), n, None),
              ("x", "w", "dy", "dx", "dw", "db", "ws"), ("x", "dy", "dx"), ("x", "w", "dy", "dx"),
              mt.head_norm_bw_workspace_bytes(d))


def test_the_binding_refuses():
    x = torch.zeros(1, 1, 4, 64)
    g = torch.zeros(1, 1, 4)
    for call in (lambda: mt.mlstm_delta_fw(x, x, x, g, g), lambda: mt.mlstm_delta_bw(x, x, x, g, g, x),
                 lambda: mt.mlstm_delta(x, x, x, g, g), lambda: mt.mlstm_delta_step(x[0], x[0], x[0], g[0], g[0]),
                 lambda: mt.head_norm_fw(x), lambda: mt.head_norm_bw(x, x), lambda: mt.head_norm(x),
                 lambda: mt.mlstm_delta_fw(x[0], x[0], x[0], g, g), lambda: mt.mlstm_delta_step(x, x, x, g, g),
                 lambda: mt.head_norm_fw(x[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mt.head_norm_fw(x.double())
