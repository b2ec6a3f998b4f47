"""Parity of the gated delta rule on many heads, where the walks give a wave
sixteen value columns of a head (256 or more workgroups of 64 columns), at
every DHQK, input type and type of H, with four and eight waves a workgroup,
with and without a second buffer (needs an MI355X).  The float64 oracle is
run on three of the heads: the first, one in the middle, the last.

Tolerances, relative to the largest magnitude of a tensor.  An output is a
chain of at most five products, each a float32 sum of at most 512 terms:
5 sqrt(512) 2^-24; a product of two operands in three truncated parts leaves
out two terms below 2^-22 of it, 5 2^-21 in all.  F32 is both, 9.2e-6.
H in bf16 reads the state in two truncated parts, off by less than 2^-15, and
P and U in two rounded ones, off by 2^-18 each and in the product left out:
H_BF16 = 2^-14 on top.  d_f adds up to 64 rows of differences whose terms do
not shrink with the result: 8 F32.  dK in bf16 has two-part operands in three
products in a row, 3 2^-15.  Storing as bf16 rounds by at most 2^-8 of the value.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import delta_fw, delta_grad  # noqa: E402
from workloads import round_to_bf16  # noqa: E402

pytestmark = pytest.mark.gpu

F32 = 5 * np.sqrt(512) * 2.0 ** -24 + 5 * 2.0 ** -21
H_BF16 = 2.0 ** -14
GATE = 8 * F32
DK_BF16 = 3 * 2.0 ** -15
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

SHAPES = [
    # B, NH, S, DHQK, DHV, inputs, state; waves a workgroup
    (16, 16, 70, 64, 64, "f32", True),       # four
    (16, 16, 150, 64, 128, "f32", False),    # eight, more threads than pieces of a tile
    (13, 20, 200, 64, 64, "bf16", True),     # four, heads not a multiple of eight
    (16, 16, 129, 64, 256, "bf16", False),   # eight
    (16, 16, 200, 128, 64, "bf16", True),    # four
    (10, 9, 131, 128, 192, "bf16", False),   # four: 192 columns
    (16, 16, 150, 128, 128, "bf16", True),   # eight
    (8, 17, 65, 128, 128, "f32", True),      # four
    (16, 16, 97, 128, 128, "f32", False),    # eight
    (4, 8, 200, 256, 512, "bf16", True),     # four
    (8, 8, 150, 256, 512, "bf16", True),     # eight
    (8, 8, 193, 256, 512, "bf16", False),
    (16, 16, 1, 256, 64, "bf16", True),      # four, one token
    (4, 8, 70, 256, 512, "f32", False),      # four
    (8, 8, 97, 256, 512, "f32", True),       # eight
    (6, 8, 64, 256, 384, "f32", True),       # four, whole chunks
]


@pytest.fixture(scope="module")
def mt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import xlstm_mlstm_chunkwise_amd as m
    m.lib()
    return m


def _dev(x, kind="f32"):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=TYPES[kind])


def _draw(B, NH, S, DK, DV, kind, state):
    rng = np.random.default_rng(1000 * B + S + DK + DV)

    def normal(*shape):
        x = rng.standard_normal(shape, dtype=np.float32)
        return round_to_bf16(x)[0] if kind == "bf16" else x

    k = rng.standard_normal((B, NH, S, DK), dtype=np.float32)
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=normal(B, NH, S, DK), k=round_to_bf16(k)[0] if kind == "bf16" else k, v=normal(B, NH, S, DV),
                i=rng.standard_normal((B, NH, S), dtype=np.float32),
                f=(1.0 + 5.0 * rng.random((B, NH, S))).astype(np.float32),
                C0=(0.3 * rng.standard_normal((B, NH, DK, DV), dtype=np.float32)) if state else None,
                dH=round_to_bf16(rng.standard_normal((B, NH, S, DV), dtype=np.float32))[0],
                dC=rng.standard_normal((B, NH, DK, DV), dtype=np.float32))


def _heads(B, NH):
    return np.array([0, B * NH // 2, B * NH - 1])


def _pick(x, heads):
    return None if x is None else x.reshape((-1,) + x.shape[2:])[heads].astype(np.float64)


def _close(got, ref, heads, rel, what):
    assert torch.isfinite(got).all(), what
    bf16 = got.dtype == torch.bfloat16
    got = got.flatten(0, 1)[torch.from_numpy(heads).cuda()].double().cpu().numpy()
    limit = rel * np.abs(ref).max() + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0)
    over = float((np.abs(got - ref) - limit).max())
    assert over <= 0, f"{what}: {over} over, largest {np.abs(ref).max()}"


@pytest.mark.parametrize("B,NH,S,DK,DV,kind,state", SHAPES)
def test_forward(mt, B, NH, S, DK, DV, kind, state):
    assert B * NH * DV // 64 >= 256
    x, heads = _draw(B, NH, S, DK, DV, kind, state), _heads(B, NH)
    args = [_dev(x[n], kind) for n in ("q", "k", "v")] + [_dev(x[n]) for n in ("i", "f")]
    C0 = _dev(x["C0"]) if state else None
    Hr, Cr = delta_fw(*[_pick(x[n], heads) for n in ("q", "k", "v", "i", "f")], _pick(x["C0"], heads))
    first = None
    for hkind in ("f32", "bf16"):
        H, C = mt.mlstm_delta_fw(*args, C0, h_dtype=TYPES[hkind])
        _close(H, Hr, heads, F32 + (H_BF16 if hkind == "bf16" else 0.0), "H " + hkind)
        _close(C, Cr, heads, F32, "C")
        assert first is None or torch.equal(first, C)
        first = C


@pytest.mark.parametrize("B,NH,S,DK,DV,kind,state", SHAPES)
def test_backward(mt, B, NH, S, DK, DV, kind, state):
    x, heads = _draw(B, NH, S, DK, DV, kind, state), _heads(B, NH)
    args = [_dev(x[n], kind) for n in ("q", "k", "v")] + [_dev(x[n]) for n in ("i", "f")]
    C0 = _dev(x["C0"]) if state else None
    r = delta_grad(*[_pick(x[n], heads) for n in ("q", "k", "v", "i", "f", "dH")], _pick(x["C0"], heads),
                   _pick(x["dC"], heads) if state else None)
    for hkind in ("f32", "bf16"):
        g = mt.mlstm_delta_bw(*args, _dev(x["dH"], hkind), C0, _dev(x["dC"]) if state else None, state_grads=True)
        for n in ("dQ", "dK", "dV", "d_i", "d_f", "dC0"):
            rel = GATE if n == "d_f" else F32 + DK_BF16 if n == "dK" and kind == "bf16" else F32
            _close(g[n], r[n], heads, rel, n + " " + hkind)


def test_gates_at_their_limits(mt):
    """Closed and open gates at a chunk's start, inside and at its end, past a
    document's end, on 256 x 512 heads with float32 H."""
    B, NH, S, DK, DV = 4, 8, 200, 256, 512
    x, heads = _draw(B, NH, S, DK, DV, "bf16", True), _heads(B, NH)
    x["f"][..., [0, 17, 18, 63, 64, 127, 150]] = -np.inf
    x["f"][..., [5, 65, 130]] = np.inf
    x["i"][..., [3, 64, 100]] = -np.inf
    x["i"][..., [4, 65, 101]] = np.inf
    args = [_dev(x[n], "bf16") for n in ("q", "k", "v")] + [_dev(x[n]) for n in ("i", "f")]
    C0, dC, picked = _dev(x["C0"]), _dev(x["dC"]), [_pick(x[n], heads) for n in ("q", "k", "v", "i", "f")]
    Hr, Cr = delta_fw(*picked, _pick(x["C0"], heads))
    H, C = mt.mlstm_delta_fw(*args, C0)
    _close(H, Hr, heads, F32, "H")
    _close(C, Cr, heads, F32, "C")
    r = delta_grad(*picked, _pick(x["dH"], heads), _pick(x["C0"], heads), _pick(x["dC"], heads))
    g = mt.mlstm_delta_bw(*args, _dev(x["dH"], "f32"), C0, dC, state_grads=True)
    for n in ("dQ", "dK", "dV", "d_i", "d_f", "dC0"):
        _close(g[n], r[n], heads, GATE if n == "d_f" else F32 + DK_BF16 if n == "dK" else F32, n)
    assert (g["d_f"][..., [0, 17, 18, 63, 64, 127, 150]] == 0).all()
    assert (g["d_i"][..., [3, 64, 100, 4, 65, 101]] == 0).all()


def test_equal_bits_and_rows_behind(mt):
    """Two calls give equal bits with any workspace contents, and nothing is
    written behind H's last row (float32 H, 256 x 512 heads: one buffer)."""
    B, NH, S, DK, DV = 4, 8, 77, 256, 512
    x = _draw(B, NH, S, DK, DV, "bf16", True)
    args = [_dev(x[n], "bf16") for n in ("q", "k", "v")] + [_dev(x[n]) for n in ("i", "f")]
    C0, dH = _dev(x["C0"]), _dev(x["dH"])
    desc = mt.make_delta_desc(B, NH, S, DK, DV)
    H, C = mt.mlstm_delta_fw(*args, C0)
    big = torch.full((H.numel() + 4096,), 7.0, device="cuda")
    ws = torch.full((mt.delta_fw_workspace_bytes(desc),), 255, dtype=torch.uint8, device="cuda")
    H2, C2 = mt.mlstm_delta_fw(*args, C0, out=big[:H.numel()].view(H.shape), workspace=ws)
    assert torch.equal(H, H2) and torch.equal(C, C2) and (big[H.numel():] == 7.0).all()
    g = mt.mlstm_delta_bw(*args, dH, C0, state_grads=True)
    ws = torch.full((mt.delta_bw_workspace_bytes(desc),), 255, dtype=torch.uint8, device="cuda")
    g2 = mt.mlstm_delta_bw(*args, dH, C0, state_grads=True, workspace=ws)
    assert all(torch.equal(g[n], g2[n]) for n in g)
