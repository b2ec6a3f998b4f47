"""Tensors of more than 2^31 values: the convolution and the scan at their end
(needs an MI355X).  Everything in front of the last tokens is zero, so that the
rows at the end, the final states and the sums are those of the last tokens
alone, up to the rounding of sums in another order.

Tolerance: both sides are float32 walks of the same 100 tokens, cut into other
pieces; each is within 100 steps of four roundings (400 2^-24 = 2.4e-5) of the
exact one relative to the magnitudes, and 1e-4 of the largest value leaves both
two of that.  bf16 results may round to the other neighbour: 2^-7 of the value."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

S, D, N, TAIL = (1 << 20) + 77, 2048, 16, 100


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of GPU memory")
    return m


def _near(got, want, what):
    got, want = got.float(), want.float()
    limit = 1e-4 * want.abs().max() + (2.0 ** -7 * want.abs() if what[0] == "b" else 0.0)
    assert ((got - want).abs() <= limit).all(), what


def _tensors():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    long, tail = {}, {}
    for n, cols in (("x", D), ("dt", D), ("z", D), ("dy", D), ("B", N), ("C", N)):
        tail[n] = torch.randn((1, TAIL, cols), generator=g, device="cuda").to(torch.bfloat16)
        long[n] = torch.zeros((1, S, cols), dtype=torch.bfloat16, device="cuda")
        long[n][:, -TAIL:] = tail[n]
    return long, tail, -torch.exp(torch.randn((D, N), generator=g, device="cuda")), torch.randn((D, 4), generator=g, device="cuda")


def test_scan_and_convolution(mt):
    long, tail, A, w = _tensors()

    def scan(t):
        return mt.selective_scan_fw(t["x"], t["dt"], A, t["B"], t["C"], None, t["z"])

    (y, h), (y1, h1) = scan(long), scan(tail)
    _near(y[:, -TAIL:], y1, "b y")
    _near(h, h1, "h")
    assert not y[:, :-TAIL].any()
    del y

    def grads(t):
        return mt.selective_scan_bw(t["x"], t["dt"], A, t["B"], t["C"], t["dy"], None, t["z"])

    r, r1 = grads(long), grads(tail)
    for n in ("dx", "ddt", "dz", "dB", "dC"):
        _near(r[n][:, -TAIL:], r1[n], "b " + n)
    for n in ("dA", "dD", "dbias"):
        _near(r[n], r1[n], n)
    assert not r["dz"][:, :-TAIL].any()
    del r

    def conv(t):
        return mt.causal_conv_fw(t["x"], w)

    (y, s), (y1, s1) = conv(long), conv(tail)
    assert torch.equal(y[:, -TAIL:], y1) and torch.equal(s, s1) and not y[:, :-TAIL].any()
    c, c1 = (mt.causal_conv_bw(t["x"], w, t["dy"]) for t in (long, tail))
    assert torch.equal(c["dx"][:, -TAIL:], c1["dx"]) and not c["dx"][:, :-TAIL - 3].any()
    for n in ("dw", "db"):
        _near(c[n], c1[n], n)
