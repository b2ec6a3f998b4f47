"""Dropout (mlstm_dropout and the autograd function) against the oracle's
generator (needs an MI355X).  Which values are dropped has to agree exactly; a
kept value takes the rounding of 1 / (1 - p), of the product and of the sum with
the residual, and of a bf16 result."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_bounds import U, close  # noqa: E402
from oracle import dropout, kept  # noqa: E402
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


def _draw(seed, shape, kind):
    v = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    v = round_to_bf16(v)[0] if kind == "bf16" else v
    return v, torch.from_numpy(v).to(device="cuda", dtype=TYPES[kind])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1,), (3,), (4,), (5,), (7, 9), (8,), (2, 100, 3), (64, 257), (3, 41, 96), (1 << 18,)])
def test_against_the_oracle(mt, shape, kind):
    x, xd = _draw(1, shape, kind)
    r, rd = _draw(2, shape, kind)
    for p, seed, offset in ((0.1, 3, 0), (0.5, 2 ** 64 - 1, 2 ** 63 + 5), (0.9, -7, 11), (0.0, 1, 1), (1 - 2.0 ** -20, 5, 6)):
        for res, resd in ((None, None), (r, rd)):
            y = mt.dropout_fw(xd, p, seed, offset, residual=resd)
            ref = dropout(x, p, seed % 2 ** 64, offset, res)
            big = np.abs(x) / (1 - p) + (0 if res is None else np.abs(res))
            close(y, ref, 3 * U * big, "y", kind)
            if res is None:
                k = kept(x.size, p, seed % 2 ** 64, offset).reshape(shape)
                assert ((y == 0).cpu().numpy() == (~k | (x == 0))).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_odd_places_and_in_place(mt, kind):
    x, xd = _draw(5, (1001,), kind)
    want = mt.dropout_fw(xd, 0.3, 9)
    big = torch.full((1100,), 7.0, dtype=TYPES[kind], device="cuda")
    for at in (1, 8, 16):
        src = torch.cat([big[:at], xd])[at:]
        out = big[at:at + 1001]
        assert torch.equal(mt.dropout_fw(src, 0.3, 9, out=out), want)
        assert (big[at + 1001:] == 7.0).all() and (big[:at] == 7.0).all()
        big.fill_(7.0)
    y = xd.clone()
    assert torch.equal(mt.dropout_fw(y, 0.3, 9, out=y), want)
    r = xd.clone()
    assert torch.equal(mt.dropout_fw(xd, 0.3, 9, residual=r, out=r), mt.dropout_fw(xd, 0.3, 9, residual=xd))


def test_a_dropped_value_may_be_anything(mt):
    x, xd = _draw(7, (4096,), "f32")
    k = torch.from_numpy(kept(4096, 0.5, 1)).cuda()
    xd[~k] = float("nan")
    assert torch.isfinite(mt.dropout_fw(xd, 0.5, 1)).all()


def test_more_than_a_grid(mt):
    """More values than one pass of the largest grid has: the same generator, counted on."""
    n = (1 << 31) + 12345
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = mt.dropout_fw(x, 0.5, 21, 22)
    del x
    blocks = np.r_[0, 1, (1 << 29) - 1, 1 << 29, (n - 1) // 4]
    from oracle import philox_words
    words = philox_words(blocks, 21, 22)
    for b, w in zip(blocks, words):
        got = y[4 * b:min(4 * b + 4, n)].float().cpu().numpy()
        assert (got == np.where(w[:len(got)] >= 2 ** 31, 2.0, 0.0)).all(), b


def test_seed_in_device_memory(mt):
    """Read when the kernel runs; a graph replayed with other seeds drops others."""
    x, xd = _draw(11, (5000,), "f32")
    seed = torch.tensor([123456789012345, 42], device="cuda")
    assert torch.equal(mt.dropout_fw(xd, 0.2, seed), mt.dropout_fw(xd, 0.2, 123456789012345, 42))
    out = torch.empty_like(xd)
    mt.dropout_fw(xd, 0.2, seed, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mt.dropout_fw(xd, 0.2, seed, out=out)
    for s, o in ((1, 2), (3, -4), (2 ** 62, 9)):
        seed.copy_(torch.tensor([s, o]))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mt.dropout_fw(xd, 0.2, s, o))


@pytest.mark.parametrize("on_device", [False, True])
def test_autograd(mt, on_device):
    x, xd = _draw(13, (6, 50, 9), "bf16")
    r, rd = _draw(14, (6, 50, 9), "bf16")
    dy, dyd = _draw(15, (6, 50, 9), "bf16")
    xd.requires_grad_(True)
    rd.requires_grad_(True)
    seed, offset = (torch.tensor([77, 5], device="cuda"), 0) if on_device else (77, 5)
    y = mt.dropout(xd, 0.25, seed, offset, residual=rd)
    # a gradient that is not contiguous
    dx, dr = torch.autograd.grad(y, [xd, rd], dyd.transpose(0, 2).contiguous().transpose(0, 2), retain_graph=True)
    close(y, dropout(x, 0.25, 77, 5, r), 3 * U * (np.abs(x) * 4 / 3 + np.abs(r)), "y", "bf16")
    close(dx, dropout(dy, 0.25, 77, 5), 2 * U * np.abs(dy) * 4 / 3, "dx", "bf16")
    assert torch.equal(dr, dyd)
    if on_device:
        seed.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            torch.autograd.grad(y, [xd], dyd)


def test_refusals_on_the_gpu(mt):
    x = torch.zeros(10, 4, device="cuda")
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(mt.MlstmError):
            mt.dropout_fw(x, p, 1)
    for call in (lambda: mt.dropout_fw(x.t(), 0.1, 1), lambda: mt.dropout_fw(x, 0.1, 2 ** 64), lambda: mt.dropout_fw(x, 0.1, 1, -2 ** 63 - 1),
                 lambda: mt.dropout_fw(x, 0.1, 1, residual=x[:5]), lambda: mt.dropout_fw(x, 0.1, torch.zeros(3, dtype=torch.int64, device="cuda")),
                 lambda: mt.dropout_fw(x, 0.1, torch.zeros(2, dtype=torch.int64, device="cuda"), 3), lambda: mt.dropout_fw(x, 0.1, 1, residual=x.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mt.dropout_fw(x.double(), 0.1, 1), lambda: mt.dropout_fw(x, 0.1, 1, residual=x.bfloat16()),
                 lambda: mt.dropout_fw(x, 0.1, torch.zeros(2, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    assert mt.dropout_fw(x[:0], 0.1, 1).shape == (0, 4)


def test_out_in_place_or_apart(mt):
    store = torch.ones(30, device="cuda")
    for out, res in ((store[4:24], None), (store[10:], store[:20])):
        with pytest.raises(ValueError):
            mt.dropout_fw(store[:20], 0.5, 1, residual=res, out=out)
    x = store[:20]
    assert mt.dropout_fw(x, 0.5, 1, out=store[:20].view(20)).data_ptr() == x.data_ptr()
