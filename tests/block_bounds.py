"""Bounds of the scan's float32 rounding errors, from the oracle's own
recurrences.

Every output is a sum of products of the inputs, the steps d, the decays a and
the gate, so an error of at most e_f in every factor f of a product is at most
prod (1 + e_f) - 1 of the product, and the output is off by at most

    walk(|inputs| (1 + errors)) - walk(|inputs|).

Factors, u = 2^-24 (half a step of float32):
  d   e^-|x| has an argument off by |x| times three roundings (the product, the
      constant, the sum with the bias) and its instruction two: (3 |x| + 2) u.
      The quotient s and the polynomial take eight more, the sum with max(x, 0)
      one: (3 |x| + 12) u of d.
  a   exp(d A): the exponent d |A| is off by its three roundings and by d's
      error, and a state that is carried over a chunk by the sum of d also by
      one rounding a token of that sum, S u; the instruction, the product with
      the state and the sum behind it take four.
  gate  as d: (3 |z| + 12) u; its slope is formed of four such factors.
  B, C  the sum over N states: N + 4 roundings.
  dy, dB, dC, dD, dA: sums over channels or tokens in runs: R roundings.
"""
import numpy as np

from oracle.mlstm_block import _prepare, scan_walk, scan_walk_grad, silu_slope

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _size(x):
    """|x| of an exponential's argument: behind 200 there is nothing left of the result."""
    return np.minimum(np.abs(x), 200.0)


def _errors(pre, d, A, z, S, N):
    ed = (3 * _size(pre) + 12) * U
    ea = 4 * U + np.abs(d[..., None] * A) * ((3 + S) * U + ed[..., None])
    eg = 0.0 if z is None else (3 * np.abs(np.asarray(z, np.float64)) + 12) * U
    return ed, ea, eg, (N + 4) * U


def scan_bounds(kw, dy=None, dh=None):
    """Bounds of y and h and, with dy, of every gradient, as a dict."""
    x, z = np.asarray(kw["x"], np.float64), kw.get("z")
    S, N = x.shape[1], kw["A"].shape[1]
    d, a, x, Bm, Cm, A, D, gate, pre, h0 = _prepare(*(kw.get(n) for n in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")))
    ed, ea, eg, en = _errors(pre, d, A, z, S, N)
    slope = np.ones(x.shape) if z is None else np.abs(silu_slope(z))
    # a slope near its zero is a difference of terms up to 1 + |z|
    wide = np.ones(x.shape) if z is None else slope + 0.3 * (1 + np.abs(z))
    plain = [d, a, np.abs(x), np.abs(Bm), np.abs(Cm), np.abs(D), np.abs(gate), np.abs(h0)]
    more = [d * (1 + ed), a * (1 + ea), plain[2] * (1 + 2 * U), plain[3] * (1 + en), plain[4] * (1 + en), plain[5] * (1 + 2 * U),
            plain[6] * (1 + eg), plain[7]]
    lo, hi = scan_walk(*plain), scan_walk(*more)
    out = dict(y=hi[0] - lo[0], h=hi[1] - lo[1])
    if dy is None:
        return out
    R = 300 + S + x.shape[-1] / 64                       # roundings of a long sum
    dy, dh = np.abs(np.asarray(dy, np.float64)), np.zeros(h0.shape) if dh is None else np.abs(np.asarray(dh, np.float64))

    def grads(f, slope, dy):
        d, a, x, Bm, Cm, D, gate, h0 = f
        return scan_walk_grad(d, a, x, Bm, Cm, np.abs(A), D, gate, slope, dy, h0, dh)

    lo, hi = grads(plain, slope, dy), grads(more, slope + wide * (4 * eg + 8 * U), dy * (1 + 4 * U))
    sums = {"dA", "dB", "dC", "dD"}
    b = {n: hi[n] - lo[n] + hi[n] * (R * U if n in sums else 0.0) for n in lo}
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-pre))
    es = (3 * _size(pre) + 12) * U
    b["ddt"] = b["dd"] * sig + hi["dd"] * sig * es
    b["dbias"] = b["ddt"].sum((0, 1)) + (hi["dd"] * sig).sum((0, 1)) * R * U
    b.pop("dd")
    return {**out, **b}


def close(got, ref, bound, what, kind="f32"):
    """got within the bound and its own rounding of ref."""
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    limit = bound + HALF_STEP[kind] * (np.abs(ref) + bound) + 2.0 ** -126
    over = np.abs(got - ref) - limit
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max()} over, {(np.abs(got - ref) / limit).max()} of the limit"
