"""The head norm's weight and bias gradients where the heads are so many that
the partial sums need more than one round of workgroups (needs an MI355X)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROW = 4 * 512 ** 0.5 * 2.0 ** -24


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("NH,D", [((1 << 18) + 3, 512), ((1 << 21) + 5, 64), (65536, 512), (65537, 512)])
def test_one_row_a_head(mt, NH, D):
    """One row a head: dbias is dy, and dweight is dy n with n = y of a norm
    without weight and bias.  Each of the two evaluations of n is a chain of
    four float32 sums of at most 512 terms, off by ROW of the largest n, and
    the product rounds by half a step."""
    g = torch.Generator(device="cuda").manual_seed(NH)
    x = torch.empty(1, NH, 1, D, device="cuda").normal_(generator=g)
    dy = torch.empty(1, 1, NH, D, device="cuda").normal_(generator=g)
    n = mt.head_norm_fw(x)
    for weight in (None, torch.full((NH, D), 2.0, device="cuda")):
        dx, dw, db = mt.head_norm_bw(x, dy, weight)
        want = (dy * n)[0, 0]
        limit = 2 * ROW * n.abs().max() * dy[0, 0].abs() + 2.0 ** -23 * want.abs()
        assert torch.equal(db, dy[0, 0]) and ((dw - want).abs() <= limit).all()
        assert torch.isfinite(dx).all()
