"""Gradients that arrive at any storage offset in the backward passes of
mlstm_delta, head_norm and mlstm_chunkwise (needs an MI355X).

Autograd hands on views: behind torch.cat a gradient is a contiguous slice of a
larger one and starts at any element, while the kernels read sixteen bytes at
a time.  The values are the same, so the results have the same bits.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _leaves(kind, S=70, D=64):
    g = torch.Generator(device="cuda").manual_seed(S)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    t = torch.bfloat16 if kind == "bf16" else torch.float32
    k = normal(1, 2, S, D)
    k /= k.norm(dim=-1, keepdim=True)
    x = [normal(1, 2, S, D).to(t), k.to(t), normal(1, 2, S, D).to(t), normal(1, 2, S), normal(1, 2, S) + 4.0]
    return [a.requires_grad_(True) for a in x]


def _same_behind_a_cat(outputs, leaves, seed=5):
    """Gradients for given gradients of the outputs, direct and through
    torch.cat with one, three or five elements before each."""
    grads = [torch.randn(o.shape, generator=torch.Generator(device="cuda").manual_seed(seed + j), device="cuda").to(o.dtype)
             for j, o in enumerate(outputs())]
    want = torch.autograd.grad(outputs(), leaves, grads)
    for before in (1, 3, 5):
        cats = [torch.cat([torch.zeros(before, device="cuda", dtype=o.dtype), o.flatten()]) for o in outputs()]
        wide = [torch.cat([torch.ones(before, device="cuda", dtype=d.dtype), d.flatten()]) for d in grads]
        got = torch.autograd.grad(cats, leaves, wide)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), before


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_delta(mt, kind):
    leaves = _leaves(kind)
    _same_behind_a_cat(lambda: list(mt.mlstm_delta(*leaves, h_dtype=leaves[0].dtype, return_final_state=True)), leaves)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_delta_and_norm(mt, kind):
    leaves = _leaves(kind)
    leaves.append(torch.rand(2, 64, device="cuda").requires_grad_(True))
    _same_behind_a_cat(lambda: [mt.mlstm_delta(*leaves[:5], norm_weight=leaves[5])], leaves)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_norm(mt, kind):
    leaves = [_leaves(kind)[0], torch.rand(2, 64, device="cuda").requires_grad_(True)]
    _same_behind_a_cat(lambda: [mt.head_norm(*leaves)], leaves)


@pytest.mark.parametrize("gate", ["exp", "sig"])
def test_cell(mt, gate):
    leaves = _leaves("bf16")
    _same_behind_a_cat(lambda: [mt.mlstm_chunkwise(*leaves, chunk_size=64, gate=gate)], leaves)
