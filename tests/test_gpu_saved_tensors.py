"""Gradients under hooks on saved tensors (activations kept on the host, or
copied): the bits of those without a hook, for inputs that are runs of columns
(needs an MI355X)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HOOKS = {"host": lambda: torch.autograd.graph.save_on_cpu(),
         "pinned": lambda: torch.autograd.graph.save_on_cpu(pin_memory=True),
         "copy": lambda: torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t)}


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _normal(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


@pytest.mark.parametrize("hook", list(HOOKS))
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 64, 3])
def test_convolution(mt, kind, hook, at):
    n, t = _normal(1), TYPES[kind]
    B, S, D, K = 2, 50, 64, 4
    wide, w, b = n(B, S, 2 * D + 3).to(t).requires_grad_(True), n(D, K).requires_grad_(True), n(D).requires_grad_(True)
    state, dy, ds = n(B, K - 1, D).to(t).requires_grad_(True), n(B, S, D).to(t), n(B, K - 1, D).to(t)

    def grads():
        y = mt.causal_conv(wide[..., at:at + D], w, b, state, activation="silu", return_final_state=True)
        return lambda: torch.autograd.grad(y, [wide, w, b, state], [dy, ds])

    want = grads()()
    with HOOKS[hook]():
        back = grads()
    assert all(torch.equal(g, r) for g, r in zip(back(), want))


@pytest.mark.parametrize("hook", list(HOOKS))
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 64])
def test_scan(mt, kind, hook, N):
    n, t = _normal(2), TYPES[kind]
    B, S, D = 2, 90, 70
    wide = n(B, S, 3 * D + 2 * N + 5).to(t).requires_grad_(True)
    A, Dm, bias, h0 = (v.requires_grad_(True) for v in (-torch.exp(n(D, N)), n(D), n(D), n(B, D, N)))
    dy, dh = n(B, S, D).to(t), n(B, D, N)

    def grads():
        x, dt, z, _, Bm, Cm = wide.split([D, D, D, 5, N, N], -1)
        out = mt.selective_scan(x, dt, A, Bm, Cm, Dm, z, bias, h0, return_final_state=True)
        return lambda: torch.autograd.grad(out, [wide, A, Dm, bias, h0], [dy, dh])

    want = grads()()
    with HOOKS[hook]():
        back = grads()
    assert all(torch.equal(g, r) for g, r in zip(back(), want))


@pytest.mark.parametrize("hook", list(HOOKS))
def test_dropout_with_its_seed_on_the_device(mt, hook):
    n = _normal(3)
    x, r, dy = n(5, 33).requires_grad_(True), n(5, 33).requires_grad_(True), n(5, 33)
    seed = torch.tensor([7, 8], device="cuda")

    def grads():
        y = mt.dropout(x, 0.4, seed, residual=r)
        return lambda: torch.autograd.grad(y, [x, r], dy)

    want = grads()()
    with HOOKS[hook]():
        back = grads()
    assert all(torch.equal(g, w) for g, w in zip(back(), want))


@pytest.mark.parametrize("hook", list(HOOKS))
def test_head_norm(mt, hook):
    n = _normal(4)
    x, w, b = n(2, 3, 20, 64).requires_grad_(True), n(3, 64).requires_grad_(True), n(3, 64).requires_grad_(True)
    dy = n(2, 20, 3, 64)

    def grads():
        y = mt.head_norm(x, w, b)
        return lambda: torch.autograd.grad(y, [x, w, b], dy)

    want = grads()()
    with HOOKS[hook]():
        back = grads()
    assert all(torch.equal(g, r) for g, r in zip(back(), want))
