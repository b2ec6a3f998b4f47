"""Pins of the oracle of the short causal convolution, the selective scan and
dropout on the CPU: worked values, limits, and gradients against central
differences.

Difference tolerance: a central difference with step h = 1e-5 is off by the
third derivative times h^2 / 6 (about 1e-10 here) and by 2^-52 |f| / h (about
1e-9 for |f| up to 50); 1e-7 leaves both two orders."""
import numpy as np
import pytest

from oracle import conv_fw, conv_grad, dropout, kept, philox_words, scan_fw, scan_grad


def _differences(f, args, grads, rng, keys):
    for name, key in keys:
        d = rng.standard_normal(args[name].shape)
        d /= np.linalg.norm(d)
        h = 1e-5
        diff = (f(**{**args, name: args[name] + h * d}) - f(**{**args, name: args[name] - h * d})) / (2 * h)
        assert abs(diff - (grads[key] * d).sum()) < 1e-7, name


def test_conv_worked():
    x = np.array([1.0, 2.0, 3.0]).reshape(1, 3, 1)
    y, s = conv_fw(x, np.array([[10.0, 1.0]]), np.array([0.5]), np.array([[[7.0]]]), act=False)
    assert np.allclose(y.ravel(), [71.5, 12.5, 23.5]) and s.ravel() == [3.0]
    y, s = conv_fw(x[:, :1], np.array([[5.0, 3.0, 2.0]]), state=np.array([[[1.0], [4.0]]]), act=False)
    assert y.ravel() == [19.0] and (s.ravel() == [4.0, 1.0]).all()
    assert np.allclose(conv_fw(np.zeros((1, 1, 1)), np.ones((1, 2)), np.array([2.0]))[0], 2 / (1 + np.exp(-2.0)))


@pytest.mark.parametrize("S,K,act", [(1, 2, True), (2, 4, True), (7, 3, False), (5, 4, True)])
def test_conv_gradients_against_differences(S, K, act):
    rng = np.random.default_rng(S + K)
    args = dict(x=rng.standard_normal((2, S, 3)), w=rng.standard_normal((3, K)), bias=rng.standard_normal(3),
                state=rng.standard_normal((2, K - 1, 3)))
    dy, ds = rng.standard_normal((2, S, 3)), rng.standard_normal((2, K - 1, 3))

    def f(**kw):
        y, s = conv_fw(act=act, **kw)
        return (dy * y).sum() + (ds * s).sum()

    g = conv_grad(dy=dy, dstate=ds, act=act, **args)
    _differences(f, args, g, rng, (("x", "dx"), ("w", "dw"), ("bias", "db"), ("state", "dstate")))


def _scan(seed, S, D=3, N=2, B=2):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    return dict(x=n((B, S, D)), dt=n((B, S, D)), A=-np.exp(n((D, N))), Bm=n((B, S, N)), Cm=n((B, S, N)), D=n(D),
                z=n((B, S, D)), dt_bias=n(D), h0=n((B, D, N))), rng


def test_scan_worked():
    # softplus(dt) = ln 2 at dt = 0: with A = -1 the decay is 1/2, and with x = 1 / ln 2 a write adds B
    one = np.ones((1, 2, 1))
    y, h = scan_fw(one / np.log(2.0), 0 * one, -np.ones((1, 1)), 3 * one, 2 * one, h0=np.full((1, 1, 1), 8.0))
    assert np.allclose(y.ravel(), [14.0, 13.0]) and np.allclose(h, 6.5)
    y2, _ = scan_fw(one / np.log(2.0), 0 * one, -np.ones((1, 1)), 3 * one, 2 * one, D=np.array([np.log(2.0)]), h0=np.full((1, 1, 1), 8.0))
    assert np.allclose(y2, y + 1.0)


def test_a_token_without_a_step_leaves_the_state():
    a, _ = _scan(1, 4)
    a["dt"][:, 2] = -np.inf
    y, h = scan_fw(**a)
    rest = {n: (np.delete(v, 2, 1) if n in ("x", "dt", "Bm", "Cm", "z") else v) for n, v in a.items()}
    y2, h2 = scan_fw(**rest)
    assert np.allclose(h, h2) and np.allclose(np.delete(y, 2, 1), y2)


@pytest.mark.parametrize("S,gated", [(1, True), (4, False), (6, True)])
def test_scan_gradients_against_differences(S, gated):
    args, rng = _scan(3 + S, S)
    if not gated:
        args["z"] = None
    dy, dh = rng.standard_normal(args["x"].shape), rng.standard_normal(args["h0"].shape)

    def f(**kw):
        y, h = scan_fw(**kw)
        return (dy * y).sum() + (dh * h).sum()

    g = scan_grad(dy=dy, dh=dh, **args)
    keys = [("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("D", "dD"), ("dt_bias", "dbias"), ("h0", "dh0")]
    _differences(f, args, g, rng, keys + ([("z", "dz")] if gated else []))


def test_generator_known_answers():
    """Published test vectors of Philox 4x32 with ten rounds."""
    assert [hex(w) for w in philox_words([0], 0, 0)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    ones = philox_words([2 ** 64 - 1], 2 ** 64 - 1, 2 ** 64 - 1)[0]
    assert [hex(w) for w in ones] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]
    pi = philox_words([0x85A308D3243F6A88], 0x299F31D0A4093822, 0x0370734413198A2E)[0]
    assert [hex(w) for w in pi] == ["0xd16cfe09", "0x94fdcceb", "0x5001e420", "0x24126ea1"]


def test_dropout_shares_and_mean():
    n, p = 1 << 16, 0.3
    k = kept(n, p, 5, 6)
    # binomial: six standard deviations of sqrt(p (1 - p) / n) = 0.0018
    assert abs(k.mean() - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5
    assert kept(n, 0.0, 5).all() and (kept(n, 0.5, 5) != kept(n, 0.5, 5, 1)).any()
    x = np.ones(n)
    assert abs(dropout(x, p, 5, 6).mean() - 1) < 0.02 and np.allclose(dropout(x, p, 5, 6, x) - 1, dropout(x, p, 5, 6))
