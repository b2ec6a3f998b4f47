"""The input gate's gradient where the gate is nearly open or nearly closed,
against the float64 oracle, row by row (needs an MI355X).

d_i_t = b (1 - b) dU_t . r_t with r_t = u_t / b.  b and 1 - b are taken out, so
that a row counts by its own digits: x_t = d_i_t / (b (1 - b)) of a row is off
by at most REL of the largest |x| (1 + 2^-21 for b, 1 - b and the two products
around them, each half a step or the few of an exponential).

REL: dU and r are float32 sums of at most 512 terms behind chains of five
products, 5 sqrt(512) 2^-24 of the largest; a product of two three-part
operands leaves out terms below 2^-21 of it, five times; together
6.8e-6 + 2.4e-6 for each of the two factors of the scalar product.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import delta_grad  # noqa: E402
from workloads import round_to_bf16  # noqa: E402

pytestmark = pytest.mark.gpu

REL = 2 * (5 * np.sqrt(512) * 2.0 ** -24 + 5 * 2.0 ** -21) + 2.0 ** -21
S = 150


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _draw(seed, DK, DV, kind):
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((1, 2, S, DK))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    x = [rng.standard_normal((1, 2, S, DK)), k, rng.standard_normal((1, 2, S, DV))]
    dH = rng.standard_normal((1, 2, S, DV))
    x, dH = [a.astype(np.float32) for a in x], dH.astype(np.float32)
    if kind == "bf16":
        x, dH = [round_to_bf16(a)[0] for a in x], round_to_bf16(dH)[0]
    i = rng.standard_normal((1, 2, S)).astype(np.float32)
    f = (1.0 + 5.0 * rng.random((1, 2, S))).astype(np.float32)
    return x, i, f, dH, (0.3 * rng.standard_normal((1, 2, DK, DV))).astype(np.float32), rng


def _check(mt, kind, x, i, f, dH, C0, rows):
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    q, k, v, h = (torch.from_numpy(a).to("cuda", t) for a in (*x, dH))
    got = mt.mlstm_delta_bw(q, k, v, torch.from_numpy(i).cuda(), torch.from_numpy(f).cuda(), h, torch.from_numpy(C0).cuda())
    want = delta_grad(*x, i, f, dH, C0)["d_i"]
    z = i.astype(np.float64)
    scale = 1.0 / (1.0 + np.exp(-z)) / (1.0 + np.exp(z))
    a, b = got["d_i"].double().cpu().numpy() / scale, want / scale
    off, largest = float(np.abs(a - b)[..., rows].max()), float(np.abs(b).max())
    assert off <= REL * largest, f"{off / largest} of the largest"


@pytest.mark.parametrize("DK,DV,kind", [(64, 64, "bf16"), (128, 192, "bf16"), (256, 128, "bf16"), (64, 128, "f32"), (256, 64, "f32")])
def test_nearly_open(mt, DK, DV, kind):
    """i up to 30: 1 - b is down to 1e-13, far below b's last digit."""
    x, i, f, dH, C0, rng = _draw(DK + DV, DK, DV, kind)
    i[..., ::3] = 5.0 + 25.0 * rng.random(i[..., ::3].shape)
    _check(mt, kind, x, i, f, dH, C0, slice(None))


@pytest.mark.parametrize("DK,DV,kind", [(64, 64, "bf16"), (128, 192, "bf16"), (256, 128, "bf16"), (64, 128, "f32"), (256, 64, "f32")])
def test_nearly_closed(mt, DK, DV, kind):
    """i down to -68: b^2 is far below the smallest float32 value, b's own
    third parts (2^-16 b and the products with them) are not yet."""
    x, i, f, dH, C0, rng = _draw(DK + DV + 1, DK, DV, kind)
    i[..., ::3] = -68.0 + 48.0 * rng.random(i[..., ::3].shape)
    _check(mt, kind, x, i, f, dH, C0, slice(None))


def test_closed_and_almost(mt):
    """Down to i = -120, where b is zero in float32.  dV and U carry b, in parts
    of eight bits: with b below 2^-110 their last parts and then their middle
    ones go below the smallest normal value, 2^-126, and the first keeps
    2^-7; two products (T with dU, T with r, whose other terms at most double
    them) make 4 2^-7 of |dU| |r|, and what is below 2^-126 may be lost."""
    x, i, f, dH, C0, _ = _draw(3, 64, 64, "bf16")
    i[..., 20:140] = np.linspace(-60.0, -120.0, 120)
    args = [torch.from_numpy(a).to("cuda", torch.bfloat16) for a in x] + [torch.from_numpy(a).cuda() for a in (i, f)]
    got = mt.mlstm_delta_bw(*args, torch.from_numpy(dH).to("cuda", torch.bfloat16), torch.from_numpy(C0).cuda())["d_i"]
    want = delta_grad(*x, i, f, dH, C0)
    z = i.astype(np.float64)
    b, a = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(-f.astype(np.float64)))
    du, r, C = want["dV"] / b[..., None], np.empty_like(want["dV"]), C0.astype(np.float64)
    for t in range(S):
        k = x[1][..., t, :].astype(np.float64)
        r[..., t, :] = x[2][..., t, :] - a[..., t, None] * np.matmul(k[..., None, :], C)[..., 0, :]
        C = a[..., t, None, None] * C + k[..., None] * (b[..., t, None] * r[..., t, :])[..., None, :]
    assert np.allclose((du * r).sum(-1) * b * (1.0 - b), want["d_i"])
    size = np.linalg.norm(du, axis=-1) * np.linalg.norm(r, axis=-1)
    lost = 2.0 ** -126 * (np.abs(du).sum(-1) + np.abs(r).sum(-1))
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = (np.abs(got - want["d_i"]) - 4 * 2.0 ** -7 * b * size - lost)[..., 20:140]
    assert off.max() <= 0, float(off.max())
    assert (got[i < -104.0] == 0).all()
