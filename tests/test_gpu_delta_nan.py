"""A NaN gate in the gated delta rule reaches everything that its token reaches
by the recurrence, in both forms of the walk and in the step, and nothing else
(needs an MI355X).

With a NaN in a_t or b_t the state is NaN from token t on, and the gradient of
the state at every token before t.  So H and dQ are NaN from row t on, dV and
dK before it, and both gate gradients everywhere, each being a product of one
with the other.  No tolerance enters: values are NaN, or keep their bits.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

S = 200
CHUNK = {"bf16": 64, "f32": 32}
# both forms of the walk: few heads, and 256 workgroups of 64 value columns
FORMS = [(2, 2), (64, 4)]


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _draw(B, NH, kind):
    g = torch.Generator(device="cuda").manual_seed(B + NH)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    t = torch.bfloat16 if kind == "bf16" else torch.float32
    k = normal(B, NH, S, 64)
    k /= k.norm(dim=-1, keepdim=True)
    args = [normal(B, NH, S, 64).to(t), k.to(t), normal(B, NH, S, 64).to(t), normal(B, NH, S), normal(B, NH, S) + 4.0]
    return args, 0.3 * normal(B, NH, 64, 64), normal(B, NH, S, 64).to(t)


def _others_keep_their_bits(a, b):
    assert torch.equal(a[0, 1:], b[0, 1:]) and torch.equal(a[1:], b[1:])


@pytest.mark.parametrize("B,NH", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("t", [0, 100])
def test_forget_gate_forward(mt, B, NH, kind, t):
    args, C0, _ = _draw(B, NH, kind)
    H, C = mt.mlstm_delta_fw(*args, C0)
    args[4][0, 0, t] = float("nan")
    for state in (C0, None):
        H2, C2 = mt.mlstm_delta_fw(*args, state)
        assert H2[0, 0, t:].isnan().all() and C2[0, 0].isnan().all()
    H2, C2 = mt.mlstm_delta_fw(*args, C0)
    start = t // CHUNK[kind] * CHUNK[kind]
    assert torch.equal(H2[0, 0, :start], H[0, 0, :start])
    _others_keep_their_bits(H2, H)
    _others_keep_their_bits(C2, C)


@pytest.mark.parametrize("B,NH", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_forget_gate_backward(mt, B, NH, kind):
    t = 100
    args, C0, dH = _draw(B, NH, kind)
    want = mt.mlstm_delta_bw(*args, dH, C0, state_grads=True)
    args[4][0, 0, t] = float("nan")
    g = mt.mlstm_delta_bw(*args, dH, C0, state_grads=True)
    for n, rows in (("dQ", slice(t, None)), ("dK", slice(None)), ("dV", slice(t)), ("d_i", slice(None)),
                    ("d_f", slice(None)), ("dC0", slice(None))):
        assert g[n][0, 0, rows].isnan().all(), n
        _others_keep_their_bits(g[n], want[n])


def test_forget_gate_step(mt):
    args, C0, _ = _draw(2, 2, "bf16")
    one = [a[:, :, 0].contiguous() for a in args]
    h, C = mt.mlstm_delta_step(*one, C0)
    one[4][0, 0] = float("nan")
    for state in (C0, None):
        h2, C2 = mt.mlstm_delta_step(*one, state)
        assert h2[0, 0].isnan().all() and C2[0, 0].isnan().all()
    h2, C2 = mt.mlstm_delta_step(*one, C0)
    _others_keep_their_bits(h2, h)
    _others_keep_their_bits(C2, C)


@pytest.mark.parametrize("B,NH", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("t", [0, 100])
def test_input_gate(mt, B, NH, kind, t):
    """b_t also stands in token t's own dV = b dU."""
    args, C0, dH = _draw(B, NH, kind)
    H, C = mt.mlstm_delta_fw(*args, C0)
    want = mt.mlstm_delta_bw(*args, dH, C0, state_grads=True)
    args[3][0, 0, t] = float("nan")
    H2, C2 = mt.mlstm_delta_fw(*args, C0)
    start = t // CHUNK[kind] * CHUNK[kind]
    assert H2[0, 0, t:].isnan().all() and C2[0, 0].isnan().all()
    assert torch.equal(H2[0, 0, :start], H[0, 0, :start])
    _others_keep_their_bits(H2, H)
    _others_keep_their_bits(C2, C)
    g = mt.mlstm_delta_bw(*args, dH, C0, state_grads=True)
    for n, rows in (("dQ", slice(t, None)), ("dK", slice(None)), ("dV", slice(t + 1)), ("d_i", slice(None)),
                    ("d_f", slice(None)), ("dC0", slice(None))):
        assert g[n][0, 0, rows].isnan().all(), n
        _others_keep_their_bits(g[n], want[n])


@pytest.mark.parametrize("B,NH", FORMS)
def test_first_forget_gate_without_a_state(mt, B, NH):
    """It multiplies a state of zeros, and its gradient is zero, unless it is
    NaN itself."""
    args, _, dH = _draw(B, NH, "bf16")
    assert (mt.mlstm_delta_bw(*args, dH)["d_f"][..., 0] == 0).all()
    args[4][0, 0, 0] = float("nan")
    d_f = mt.mlstm_delta_bw(*args, dH)["d_f"]
    assert d_f[0, 0].isnan().all()
    assert (d_f[0, 1:, 0] == 0).all() and (d_f[1:, :, 0] == 0).all()


def test_input_gate_step(mt):
    args, C0, _ = _draw(2, 2, "f32")
    one = [a[:, :, 0].contiguous() for a in args]
    h, C = mt.mlstm_delta_step(*one, C0)
    one[3][0, 0] = float("nan")
    h2, C2 = mt.mlstm_delta_step(*one, C0)
    assert h2[0, 0].isnan().all() and C2[0, 0].isnan().all()
    _others_keep_their_bits(h2, h)
    _others_keep_their_bits(C2, C)
