"""Pins of the gated delta rule's and the head norm's oracle on the CPU: worked
values, limits of the gates, and the gradients against central differences.

Difference tolerance: a central difference with step h = 1e-5 is off by the
third derivative times h^2 / 6 (about 1e-10 here) and by 2^-52 |f| / h (about
1e-10 for |f| up to 10); 1e-7 leaves both two orders."""
import numpy as np
import pytest

from oracle import delta_fw, delta_grad, head_norm_fw, head_norm_grad


def _draw(seed, S, DK=3, DV=4, lead=(2,)):
    rng = np.random.default_rng(seed)
    k = rng.standard_normal(lead + (S, DK))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=rng.standard_normal(lead + (S, DK)), k=k, v=rng.standard_normal(lead + (S, DV)),
                i_pre=rng.standard_normal(lead + (S,)), f_pre=rng.standard_normal(lead + (S,)) + 1.0,
                C0=rng.standard_normal(lead + (DK, DV)))


def test_two_worked_steps():
    # DHQK = DHV = 1, a = b = 1/2, s = 1: C1 = 0 + 1/2 (4 - 0) = 2;
    # C2 = 1/2 * 2 + 1/2 (1 - 1/2 * 2) = 1
    one = np.ones((2, 1))
    H, C = delta_fw(3 * one, one, np.array([[4.0], [1.0]]), np.zeros(2), np.zeros(2), qk_scale=1.0)
    assert np.allclose(H[:, 0], [6.0, 3.0]) and np.allclose(C, 1.0)


def test_full_write_replaces_what_a_key_holds():
    # b = 1, a = 1, one key: the memory returns the last value written
    x = _draw(1, 5)
    k = np.broadcast_to(x["k"][..., :1, :], x["k"].shape)
    _, C = delta_fw(x["q"], k, x["v"], np.full((2, 5), np.inf), np.full((2, 5), np.inf), x["C0"])
    got = np.matmul(np.swapaxes(C, -1, -2), k[..., 0, :, None])[..., 0]
    assert np.allclose(got, x["v"][..., -1, :])


def test_a_closed_forget_gate_clears_the_memory():
    x = _draw(2, 6)
    x["f_pre"][..., 3] = -np.inf
    H, C = delta_fw(**x)
    tail = {n: (a[..., 3:, :] if a.ndim == 3 and n in "qkv" else a[..., 3:]) for n, a in x.items() if n != "C0"}
    H2, C2 = delta_fw(**tail)
    assert np.allclose(H[..., 3:, :], H2) and np.allclose(C, C2)


@pytest.mark.parametrize("S", [1, 4, 7])
def test_delta_gradients_against_differences(S):
    x = _draw(3 + S, S)
    rng = np.random.default_rng(9)
    dH, dC = rng.standard_normal(x["v"].shape), rng.standard_normal(x["C0"].shape)

    def f(**kw):
        H, C = delta_fw(**{**x, **kw})
        return (dH * H).sum() + (dC * C).sum()

    g = delta_grad(dH=dH, dC=dC, **x)
    for name, key in (("q", "dQ"), ("k", "dK"), ("v", "dV"), ("i_pre", "d_i"), ("f_pre", "d_f"), ("C0", "dC0")):
        d = rng.standard_normal(x[name].shape)
        d /= np.linalg.norm(d)
        h = 1e-5
        diff = (f(**{name: x[name] + h * d}) - f(**{name: x[name] - h * d})) / (2 * h)
        assert abs(diff - (g[key] * d).sum()) < 1e-7, name


def test_head_norm_worked_and_gradients():
    x = np.array([1.0, 3.0, 1.0, 3.0]).reshape(1, 1, 1, 4)
    assert np.allclose(head_norm_fw(x, eps=0.0).ravel(), [-1, 1, -1, 1])
    rng = np.random.default_rng(4)
    x, w, b = rng.standard_normal((2, 3, 5, 8)), rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    y = head_norm_fw(x, w, b)
    assert y.shape == (2, 5, 3, 8)
    dy = rng.standard_normal(y.shape)
    dx, dw, db = head_norm_grad(x, dy, w)
    f = lambda x_, w_, b_: (dy * head_norm_fw(x_, w_, b_)).sum()
    for at, g in ((0, dx), (1, dw), (2, db)):
        args = [x, w, b]
        d = rng.standard_normal(g.shape)
        d /= np.linalg.norm(d)
        lo, hi = list(args), list(args)
        hi[at], lo[at] = args[at] + 1e-5 * d, args[at] - 1e-5 * d
        assert abs((f(*hi) - f(*lo)) / 2e-5 - (g * d).sum()) < 1e-7
