"""Parity of the head norm (mlstm_head_norm_fw, _bw, the autograd function and
the cells' norm_weight) against the float64 oracle (needs an MI355X).

Tolerances.  A row's mean and variance are float32 sums of D <= 512 values in
registers and lanes: sqrt(512) 2^-24 = 1.4e-6 of their terms; with the products
around them four such roundings, ROW = 5.4e-6 of the tensor's largest value.
dweight and dbias add R rows in runs: sqrt(R) 2^-24 of the largest term times
sqrt(R) terms, taken relative to sqrt(R) max|term|.  bf16 results round by 2^-8
of the value on top.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import head_norm_fw, head_norm_grad, recurrent_fw  # noqa: E402
from workloads import round_to_bf16  # noqa: E402

pytestmark = pytest.mark.gpu

ROW = 4 * np.sqrt(512) * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _dev(x, kind="f32"):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=TYPES[kind])


def _close(got, ref, limit, what):
    if got.dtype == torch.bfloat16:
        limit = limit + 2.0 ** -8 * np.abs(ref)
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    over = np.abs(got - ref) - limit
    assert over.max() <= 0, f"{what}: {over.max()} over"


def _draw(seed, B, NH, S, D, xk, yk, mean=0.3):
    rng = np.random.default_rng(seed)
    x = ((rng.standard_normal((B, NH, S, D)) + mean) * (0.1 + 2 * rng.random((B, NH, S, 1)))).astype(np.float32)
    dy = rng.standard_normal((B, S, NH, D)).astype(np.float32)
    x = round_to_bf16(x)[0] if xk == "bf16" else x
    dy = round_to_bf16(dy)[0] if yk == "bf16" else dy
    return x, dy, (1 + 0.2 * rng.standard_normal((NH, D))).astype(np.float32), rng.standard_normal((NH, D)).astype(np.float32)


@pytest.mark.parametrize("B,NH,S,D,xk,yk", [
    (1, 1, 1, 64, "f32", "f32"), (2, 3, 1, 512, "bf16", "bf16"), (1, 2, 37, 128, "bf16", "f32"),
    (3, 5, 17, 192, "f32", "bf16"), (2, 1, 65, 256, "bf16", "bf16"), (1, 4, 9, 320, "f32", "f32"),
    (2, 2, 33, 384, "bf16", "bf16"), (1, 3, 5, 448, "f32", "bf16"), (2, 2, 700, 512, "f32", "f32"),
    (1, 1, 5000, 64, "bf16", "bf16")])
@pytest.mark.parametrize("parts", ["both", "weight", "none"])
def test_forward_and_backward(mt, B, NH, S, D, xk, yk, parts):
    x, dy, w, b = _draw(S + D, B, NH, S, D, xk, yk)
    w, b = None if parts == "none" else w, b if parts == "both" else None
    wd, bd = (None if a is None else _dev(a) for a in (w, b))
    y = mt.head_norm_fw(_dev(x, xk), wd, bd, y_dtype=TYPES[yk])
    ref = head_norm_fw(x, w, b)
    _close(y, ref, ROW * np.abs(ref).max(), "y")
    dx, dw, db = mt.head_norm_bw(_dev(x, xk), _dev(dy, yk), wd)
    rx, rw, rb = head_norm_grad(x, dy, w)
    _close(dx, rx, ROW * np.abs(rx).max(), "dx")
    R = B * S
    n = np.abs(head_norm_fw(x)).max()
    _close(dw, rw, (ROW + R ** 0.5 * 2.0 ** -24) * R ** 0.5 * n * np.abs(dy).max(), "dw")
    _close(db, rb, R * 2.0 ** -24 * np.abs(dy).max(), "db")
    assert all(t is None for t in mt.head_norm_bw(_dev(x, xk), _dev(dy, yk), wd, weight_grads=False)[1:])


def test_rows_without_spread_and_far_from_zero(mt):
    """A constant row has variance 0: y is the bias, dx is bounded by 1/sqrt(eps).
    A mean 2^10 times the spread costs ten of the row's 24 bits."""
    x = np.full((1, 2, 3, 64), 5.0, np.float32)
    x[0, 1] += np.random.default_rng(1).integers(-8, 8, (3, 64)) * 0.0078125 + 3.0
    w, b = np.full((2, 64), 1.5, np.float32), np.full((2, 64), 0.25, np.float32)
    y = mt.head_norm_fw(_dev(x), _dev(w), _dev(b), eps=1e-5)
    assert (y[:, :, 0] == 0.25).all()
    ref = head_norm_fw(x, w, b, 1e-5)
    _close(y, ref, 2 ** 10 * ROW * np.abs(ref).max(), "y")
    dy = np.random.default_rng(2).standard_normal((1, 3, 2, 64)).astype(np.float32)
    rx = head_norm_grad(x, dy, w, 1e-5)[0]
    _close(mt.head_norm_bw(_dev(x), _dev(dy), _dev(w), eps=1e-5)[0], rx, 2 ** 10 * ROW * np.abs(rx).max(), "dx")


def test_no_rows(mt):
    x = torch.empty(2, 3, 0, 128, device="cuda")
    assert mt.head_norm_fw(x).shape == (2, 0, 3, 128)
    dx, dw, db = mt.head_norm_bw(x, torch.empty(2, 0, 3, 128, device="cuda"))
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


def test_equal_bits_and_nothing_behind(mt):
    x, dy, w, b = _draw(3, 2, 3, 401, 192, "bf16", "bf16")
    xd, dyd, wd, bd = _dev(x, "bf16"), _dev(dy, "bf16"), _dev(w), _dev(b)
    first = mt.head_norm_bw(xd, dyd, wd)
    ws = torch.full((mt.head_norm_bw_workspace_bytes(mt.make_head_norm_desc(2, 3, 401, 192)),), 255, dtype=torch.uint8,
                    device="cuda")
    assert all(torch.equal(a, c) for a, c in zip(first, mt.head_norm_bw(xd, dyd, wd, workspace=ws)))
    big = torch.full((dy.size + 1024,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = mt.head_norm_fw(xd, wd, bd, out=big[:dy.size].view(dyd.shape))
    assert torch.equal(y, mt.head_norm_fw(xd, wd, bd)) and (big[dy.size:] == 3.0).all()


def test_a_row_with_nan_stays_alone(mt):
    x, _, w, b = _draw(4, 1, 2, 20, 128, "f32", "f32")
    y = mt.head_norm_fw(_dev(x), _dev(w), _dev(b))
    x[0, 1, 7, 3] = np.nan
    y2 = mt.head_norm_fw(_dev(x), _dev(w), _dev(b))
    assert y2[0, 7, 1].isnan().all()
    y2[0, 7, 1] = y[0, 7, 1]
    assert torch.equal(y, y2)


def test_autograd_gives_what_is_asked_for(mt):
    x, dy, w, b = _draw(5, 2, 2, 30, 128, "f32", "f32")
    xd, wd, bd = _dev(x), _dev(w).requires_grad_(True), _dev(b)
    mt.head_norm(xd, wd, bd).backward(_dev(dy).transpose(0, 0))
    rw = head_norm_grad(x, dy, w)[1]
    _close(wd.grad, rw, ROW * 60 ** 0.5 * 20, "dw")
    xd.requires_grad_(True)
    y = mt.head_norm(xd)
    (dx,) = torch.autograd.grad(y, [xd], _dev(dy))
    rx = head_norm_grad(x, dy)[0]
    _close(dx, rx, ROW * np.abs(rx).max(), "dx")


def test_behind_the_cell(mt):
    """mlstm_chunkwise with norm_weight is the cell, then the norm (and its
    backward pass reaches the cell's inputs); without it nothing changes."""
    rng = np.random.default_rng(8)
    q, k, v = (round_to_bf16(rng.standard_normal((1, 2, 70, 64)).astype(np.float32))[0] for _ in range(3))
    i, f = rng.standard_normal((1, 2, 70)).astype(np.float32), (3 + rng.random((1, 2, 70))).astype(np.float32)
    args = [_dev(a, "bf16") for a in (q, k, v)] + [_dev(i), _dev(f)]
    w = _dev(1 + 0.2 * rng.standard_normal((2, 64))).requires_grad_(True)
    for a in args:
        a.requires_grad_(True)
    H = mt.mlstm_chunkwise(*args, chunk_size=64)
    y = mt.mlstm_chunkwise(*args, chunk_size=64, norm_weight=w)
    assert y.dtype == torch.bfloat16 and torch.equal(y, mt.head_norm_fw(H.detach(), w.detach(), y_dtype=torch.bfloat16))
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(1)).to("cuda", torch.bfloat16)
    got = torch.autograd.grad(y, args + [w], dy)
    dx, dw, _ = mt.head_norm_bw(H.detach(), dy, w.detach())
    want = torch.autograd.grad(H, args, dx)
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and torch.equal(got[-1], dw)
    with pytest.raises(ValueError):
        mt.mlstm_chunkwise(*args, chunk_size=64, norm_bias=w)


@pytest.mark.parametrize("B,NH,S,D,xk,yk", [(3, 5, 2185, 512, "bf16", "f32"), (1, 16411, 2, 512, "f32", "bf16"),
                                            (4, 8209, 1, 448, "bf16", "bf16"), (1, 3, 87391, 64, "f32", "f32")])
def test_rows_four_at_a_time(mt, B, NH, S, D, xk, yk):
    """Enough rows for four of them a lane group, heads ending inside a group."""
    x, dy, w, b = _draw(S + D, B, NH, S, D, xk, yk)
    for wd, bd in ((w, b), (None, None)):
        y = mt.head_norm_fw(_dev(x, xk), *(None if a is None else _dev(a) for a in (wd, bd)), y_dtype=TYPES[yk])
        ref = head_norm_fw(x, wd, bd)
        _close(y, ref, ROW * np.abs(ref).max(), "y")
    dx = mt.head_norm_bw(_dev(x, xk), _dev(dy, yk), _dev(w), weight_grads=False)[0]
    rx = head_norm_grad(x, dy, w)[0]
    _close(dx, rx, ROW * np.abs(rx).max(), "dx")


def test_offsets_beyond_32_bits(mt):
    """The most rows that are taken, 2^26 - 1 of 64 values: 8.6 GB of x."""
    S = (1 << 26) - 1
    x = torch.zeros(1, 1, S, 64, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(1, S, 1, 64, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x[:, :, -1001:].normal_(generator=gen)
    dy[:, -1001:].normal_(generator=gen)
    w, b = torch.full((1, 64), 1.5, device="cuda"), torch.full((1, 64), 0.25, device="cuda")
    xt, dyt = x[:, :, -1001:].contiguous(), dy[:, -1001:].contiguous()
    y = mt.head_norm_fw(x, w, b)
    assert torch.equal(y[:, -1001:], mt.head_norm_fw(xt, w, b)) and (y[:, :-1001] == 0.25).all()
    dx, dw, db = mt.head_norm_bw(x, dy, w)
    rx, rw, rb = mt.head_norm_bw(xt, dyt, w)
    assert torch.equal(dx[:, :, -1001:], rx) and (dx[:, :, :-1001] == 0).all()
    # the same 1001 terms, in other runs: each sum rounds by at most 2^-24 of the sum of their sizes
    for got, want, term in ((dw, rw, 8.0 * dyt.float().abs()), (db, rb, dyt.float().abs())):
        limit = 2 * 1001 * 2.0 ** -24 * term.sum(1)[0].max()
        assert ((got - want).abs() <= limit).all()
