"""What the backward passes read where a hook on saved tensors hands back other
tensors than the forward pass was given: copies that are contiguous where it had
a run of columns, or tensors of another type or shape.  On the CPU, with the
launch replaced by a recorder of its arguments."""
import ctypes

import pytest

import xlstm_mlstm_chunkwise_amd as mt

torch = pytest.importorskip("torch")

B, S, D, K, N = 2, 50, 64, 4, 16


@pytest.fixture
def calls(monkeypatch):
    """(entry point, arguments) of every launch, in order; nothing is launched."""
    made = []
    monkeypatch.setattr(mt, "_call", lambda where, dev, *args: made.append((where, args)))
    monkeypatch.setattr(mt, "_gpu_input", lambda x, dims, layout: x.device)
    monkeypatch.setattr(mt, "_norm_input", lambda x: x.shape)
    return made


class _Kept:
    """A pair of hooks that hands back `change` of every saved tensor, and keeps
    it, so that its memory can be looked up by address."""

    def __init__(self, change):
        self.change, self.back = change, {}

    def pack(self, t):
        return t

    def unpack(self, t):
        t = self.change(t.detach())
        self.back[t.data_ptr()] = t
        return t

    def hooks(self):
        return torch.autograd.graph.saved_tensors_hooks(self.pack, self.unpack)


def _copy(t):
    return t.clone(memory_format=torch.contiguous_format)


def _inside(kept, address, strides, shape):
    """The elements that a view's strides reach from this address lie in the tensor handed back there, and are its own."""
    t = kept.back[address]
    batch, token = strides[0] or shape[1] * shape[2], strides[1] or shape[2]
    last = (shape[0] - 1) * batch + (shape[1] - 1) * token + shape[2]
    assert last <= t.numel() and (batch, token) == t.stride()[:2], (strides, t.stride())


def test_convolution_of_a_run_of_columns(calls):
    kept = _Kept(_copy)
    xz, w = torch.randn(B, S, 2 * D, requires_grad=True), torch.randn(D, K, requires_grad=True)
    with kept.hooks():
        y = mt.causal_conv(xz[..., :D], w, activation="silu")
    torch.autograd.grad(y, [xz, w], torch.randn(B, S, D))
    (fw, _), (bw, args) = calls
    assert (fw, bw) == ("mlstm_conv_fw", "mlstm_conv_bw")
    desc = ctypes.cast(args[0], ctypes.POINTER(mt.ConvDesc)).contents
    _inside(kept, args[1], desc.x_strides, (B, S, D))


def test_scan_of_runs_of_columns(calls):
    kept = _Kept(_copy)
    wide = torch.randn(B, S, 3 * D + 4 + 2 * N, requires_grad=True)
    x, dt, z, _, Bm, Cm = wide.split([D, D, D, 4, N, N], -1)
    A = (-torch.rand(D, N)).requires_grad_(True)
    with kept.hooks():
        y = mt.selective_scan(x, dt, A, Bm, Cm, None, z)
    torch.autograd.grad(y, [wide, A], torch.randn(B, S, D))
    (fw, _), (bw, args) = calls
    assert (fw, bw) == ("mlstm_scan_fw", "mlstm_scan_bw")
    desc = ctypes.cast(args[0], ctypes.POINTER(mt.ScanDesc)).contents
    for at, strides, cols in ((1, desc.x_strides, D), (2, desc.dt_strides, D), (7, desc.z_strides, D), (4, desc.B_strides, N), (5, desc.C_strides, N)):
        _inside(kept, args[at], strides, (B, S, cols))


def test_views_stay_views_without_a_hook(calls):
    xz, w = torch.randn(B, S, 2 * D, requires_grad=True), torch.randn(D, K, requires_grad=True)
    y = mt.causal_conv(xz[..., D:], w)
    torch.autograd.grad(y, [xz, w], torch.randn(B, S, D))
    desc = ctypes.cast(calls[1][1][0], ctypes.POINTER(mt.ConvDesc)).contents
    assert tuple(desc.x_strides) == (S * 2 * D, 2 * D)


@pytest.mark.parametrize("change", [lambda t: t.to(torch.bfloat16), lambda t: t[..., :1], lambda t: t.flatten()], ids=["type", "columns", "rank"])
def test_other_types_and_shapes_are_refused(calls, change):
    x, w, b = torch.randn(B, S, D, requires_grad=True), torch.randn(D, K), torch.randn(D)
    dt, Bm, Cm, A = torch.randn(B, S, D), torch.randn(B, S, N), torch.randn(B, S, N), -torch.rand(D, N)
    with _Kept(change).hooks():
        ys = [mt.causal_conv(x, w, b), mt.selective_scan(x, dt, A, Bm, Cm, b)]
    for y in ys:
        with pytest.raises((TypeError, ValueError, IndexError)):
            torch.autograd.grad(y, [x], torch.randn(B, S, D))
    assert len(calls) == 2


def test_head_norm(calls, monkeypatch):
    """A weight of another type or shape, x as a transposed copy."""
    x, w = torch.randn(2, 3, 5, 64, requires_grad=True), torch.randn(3, 64, requires_grad=True)

    def inputs(x):
        if not x.is_contiguous():
            raise ValueError("x must be contiguous")
        return x.shape

    monkeypatch.setattr(mt, "_norm_input", inputs)
    for change in (lambda t: t.to(torch.bfloat16) if t.dim() == 2 else t, lambda t: t[:1] if t.dim() == 2 else t,
                   lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)):
        with _Kept(change).hooks():
            y = mt.head_norm(x, w)
        with pytest.raises((TypeError, ValueError)):
            torch.autograd.grad(y, [x, w], torch.randn_like(y))
    assert [where for where, _ in calls] == ["mlstm_head_norm_fw"] * 3
    calls.clear()
    y = mt.head_norm(x, w)
    torch.autograd.grad(y, [x, w], torch.randn_like(y))
    assert [where for where, _ in calls] == ["mlstm_head_norm_fw", "mlstm_head_norm_bw"]
