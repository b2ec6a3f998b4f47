"""The selective scan where the sequence is cut into chunks of states and spans
of gradients in every way that the sizes lead to: several spans in a chunk, one
chunk of several spans, spans that are chunks (needs an MI355X).  The states and
gradients that pieces hand on to each other are alive: steps from 0.0025 on keep
a state over hundreds of tokens.

Each case asserts its cut by the workspaces' sizes: the forward pass keeps a
state and a float a channel for each chunk where there are several, the backward
pass also for each span.  N = 32 and 64 have no more spans than chunks."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_bounds import U, close, scan_bounds  # noqa: E402
from oracle import scan_fw, scan_grad  # noqa: E402
from test_gpu_scan import _args, _bw, _check, _draw  # noqa: E402


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _size(*floats):
    return sum((4 * n + 255) // 256 * 256 for n in floats)


def assert_cut(mt, B, S, D, N, forward, chunks, spans):
    """Chunks of the forward pass; chunks and spans of the backward pass."""
    rows, groups = (S + 15) // 16 * 16, -(-D * N // 2048)

    def walk(chunks):
        return [B * rows * 2 * N] + ([B * chunks * D * N, B * chunks * D] if chunks > 1 else [])

    desc = mt.make_scan_desc(B, S, D, N)
    assert mt.scan_fw_workspace_bytes(desc) == _size(*walk(forward))
    handed = [B * spans * D * N, B * spans * D] if spans > 1 else []
    assert mt.scan_bw_workspace_bytes(desc) == _size(*walk(chunks), *handed, B * (rows // 8) * D * N, groups * B * S * 2 * N, B * spans * D * N,
                                                     2 * B * spans * D)


CUTS = [  # forward chunks, backward chunks, spans
    ((20, 793, 70, 16), (17, 13, 25)),     # two spans a chunk
    ((60, 250, 65, 16), (6, 4, 8)),
    ((100, 230, 66, 16), (3, 2, 4)),
    ((129, 150, 65, 16), (1, 1, 3)),       # one chunk
    ((1, 150, 65, 16), (5, 5, 5)),         # a span a chunk
    ((50, 300, 65, 32), (7, 5, 5)),
    ((3, 200, 130, 64), (5, 4, 4)),
    ((17, 333, 100, 64), (7, 6, 6)),
    ((130, 70, 65, 32), (1, 1, 1)),
    ((65, 64, 200, 64), (1, 1, 1)),        # enough workgroups for no cut at all
]


LONG = [
    ((3, 1777, 960, 16), (16, 10, 19)),    # two spans a chunk, the last chunk of one
    ((8, 2048, 4096, 16), (1, 1, 2)),      # one chunk of two spans
    ((3, 1777, 961, 32), (16, 10, 10)),
    ((1, 2500, 200, 64), (53, 40, 40)),
]


def test_the_cuts():
    import xlstm_mlstm_chunkwise_amd as m
    for shape, cut in CUTS + LONG:
        assert_cut(m, *shape, *cut)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shape,cut", CUTS)
def test_against_the_oracle(mt, shape, cut, kind):
    assert_cut(mt, *shape, *cut)
    _check(mt, *_draw(sum(shape), *shape, kind), kind)


def _walk(d, a, x, Bm, Cm, A, D, gate, slope, dy, h0, dh):
    """The recurrence and its adjoint, token by token, in the tensors' 64 bits:
    the oracle's scan_walk and scan_walk_grad on the GPU."""
    S, h, states, r = x.shape[1], h0, [h0], torch.empty_like(x)
    for t in range(S):
        h = a[:, t] * h + (d[:, t] * x[:, t])[..., None] * Bm[:, t, None]
        states.append(h)
        r[:, t] = (h * Cm[:, t, None]).sum(-1) + D * x[:, t]
    out = dict(y=r * gate, h=h, dz=dy * r * slope)
    dr, g, dA = dy * gate, dh, torch.zeros_like(A)
    dx, dd, dB, dC = torch.empty_like(x), torch.empty_like(x), torch.empty_like(Bm), torch.empty_like(Cm)
    for t in reversed(range(S)):
        g = g + dr[:, t, :, None] * Cm[:, t, None]
        dC[:, t] = (dr[:, t, :, None] * states.pop()).sum(1)
        dB[:, t] = (g * (d[:, t] * x[:, t])[..., None]).sum(1)
        s = (g * Bm[:, t, None]).sum(-1)
        g = a[:, t] * g
        w = g * states[-1]
        dA += (d[:, t, :, None] * w).sum(0)
        dd[:, t] = x[:, t] * s + (A * w).sum(-1)
        dx[:, t] = d[:, t] * s + D * dr[:, t]
    return dict(out, dx=dx, dd=dd, dA=dA, dB=dB, dC=dC, dD=(dr * x).sum((0, 1)), dh0=g)


def _exact(g, dy, dh):
    """Outputs and gradients in 64 bits, and their bounds, formed as scan_bounds
    forms them from the same errors of the factors."""
    x, dt, A, Bm, Cm, D, z, bias, h0 = (v.double() for v in _args(g))
    dy, dh, S, N = dy.double(), dh.double(), x.shape[1], A.shape[1]
    pre, sz = dt + bias, torch.sigmoid(z)
    d, gate, slope = pre.clamp(min=0) + torch.log1p(torch.exp(-pre.abs())), z * sz, sz * (1 + z * (1 - sz))
    a = torch.exp(d[..., None] * A)
    ref = _walk(d, a, x, Bm, Cm, A, D, gate, slope, dy, h0, dh)
    size = lambda v: v.abs().clamp(max=200)
    ed, eg, en = (3 * size(pre) + 12) * U, (3 * z.abs() + 12) * U, (N + 4) * U
    mag = [d, a, x.abs(), Bm.abs(), Cm.abs(), A.abs(), D.abs(), gate.abs(), slope.abs(), dy.abs(), h0.abs(), dh.abs()]
    lo = _walk(*mag)
    ea = 4 * U + d[..., None] * A.abs() * ((3 + S) * U + ed[..., None])
    wide = slope.abs() + 0.3 * (1 + z.abs())
    hi = _walk(d * (1 + ed), a * (1 + ea), mag[2] * (1 + 2 * U), mag[3] * (1 + en), mag[4] * (1 + en), mag[5], mag[6] * (1 + 2 * U),
               mag[7] * (1 + eg), mag[8] + wide * (4 * eg + 8 * U), mag[9] * (1 + 4 * U), mag[10], mag[11])
    R = 300 + S + x.shape[-1] / 64
    b = {k: hi[k] - lo[k] + (hi[k] * R * U if k in ("dA", "dB", "dC", "dD") else 0) for k in lo}
    sig = torch.sigmoid(pre)
    ref["ddt"] = ref.pop("dd") * sig
    ref["dbias"] = ref["ddt"].sum((0, 1))
    dd = hi["dd"] * sig
    b["ddt"] = b.pop("dd") * sig + dd * ed
    b["dbias"] = b["ddt"].sum((0, 1)) + dd.sum((0, 1)) * R * U
    return ref, b


def _gpu_draw(B, S, D, N):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(B + S + D + N)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")
    g = dict(x=n(B, S, D), dt=0.7 * n(B, S, D), A=-torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * n(D, N)), Bm=n(B, S, N), Cm=n(B, S, N),
             D=1 + 0.1 * n(D), z=n(B, S, D), dt_bias=-6 + 5 * torch.rand(D, generator=gen, device="cuda"), h0=0.3 * n(B, D, N))
    return g, n(B, S, D), n(B, D, N)


@pytest.mark.gpu
@pytest.mark.parametrize("shape,cut", [CUTS[1], CUTS[3], CUTS[6]])
def test_growing_states(mt, shape, cut):
    """A of either sign: products of decays up to e^5 and back to e^-5."""
    assert_cut(mt, *shape, *cut)
    kw, dy, dh = _draw(sum(shape) + 1, *shape, "f32")
    steps = np.logaddexp(0, kw["dt"] + kw["dt_bias"]).sum(1).max()
    kw["A"] = (5 / steps * np.random.default_rng(2).uniform(-1, 1, kw["A"].shape)).astype(np.float32)
    _check(mt, kw, dy, dh, "f32")


@pytest.mark.gpu
def test_the_walk_is_the_oracles(mt):
    g, dy, dh = _gpu_draw(2, 40, 24, 16)
    kw, host = {k: v.cpu().numpy() for k, v in g.items()}, (dy.cpu().numpy(), dh.cpu().numpy())
    ref, b = _exact(g, dy, dh)
    want, bounds = dict(zip("yh", scan_fw(**kw)), **scan_grad(dy=host[0], dh=host[1], **kw)), scan_bounds(kw, *host)
    assert set(ref) == set(want) == set(b) == set(bounds)
    for k in want:
        assert np.allclose(ref[k].cpu().numpy(), want[k], rtol=1e-11, atol=1e-12), k
        # (bounds are differences of sums that agree to 1e-13)
        assert np.allclose(b[k].cpu().numpy(), bounds[k], rtol=1e-5, atol=1e-11), k


@pytest.mark.gpu
@pytest.mark.parametrize("shape,cut", LONG)
def test_long_sequences(mt, shape, cut):
    """Every value against 64 bits."""
    assert_cut(mt, *shape, *cut)
    g, dy, dh = _gpu_draw(*shape)
    y, h = mt.selective_scan_fw(*_args(g))
    got = dict(y=y, h=h, **_bw(mt, g, dy, dh))
    ref, b = _exact(g, dy, dh)
    assert set(got) == set(ref)
    for k in got:
        # within the bound and the value's own rounding
        over = (got[k].double() - ref[k]).abs() - (b[k] + U * (ref[k].abs() + b[k]) + 2.0 ** -126)
        assert torch.isfinite(got[k]).all() and over.max() <= 0, (k, over.max().item())
