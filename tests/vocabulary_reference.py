"""Float64 reference of the losses over a packed vocabulary matrix and of the
embedding, on small shapes, with a bound on each output (test infrastructure).

The weights are the CPU oracle's (exact bf16 numbers); everything else is
float64 NumPy from the formulas.

Bounds, E24 = 2^-24:
* a logit is a float32 sum of K exact products: off by K E24 sum|w x|; in the
  exponent's unit (times log2(e) / T, two roundings more) by 3 E24 |l| / T;
* lse: its logits' errors weighted by p, at most their largest; a term
  2^(l2 - R) is off by a relative 2^-22 (the difference's rounding, at most a
  rounding of 2^-24 l2 weighted with p, and the exponential's own of one unit), the sum of
  them by at most 128 roundings one after the other (16 a thread, 8 to join the
  workgroup, up to 64 spans, the list), in all 2^-17 at the most; the logarithm
  and the last products 4 E24 |lse|;
* the teacher's q: 2^-19 relative (difference, exponential, at most 256
  additions of which each thread makes 12 in turn, division), log q likewise plus
  4 E24 |log q| and the teacher's scaled logits' 3 E24 |z| / T;
* loss of a row with one entry: log(1 + S'/e), whose derivative by the logits'
  errors is 1 - p; of other rows: the errors of log q and log p weighted by q;
* d = T (p - q): a relative error of p by the errors of l and lse, q's, and half
  a bf16 step of d or, where p is kept without the division, of p (2^-8);
* dx: d's errors times |W|, N E24 of the sum of the terms' magnitudes, and the
  last rounding.
"""
from __future__ import annotations

import numpy as np

from tests.rows_reference import E24, bf16, rounded, weights
from workloads import make_codes, make_scales


def draw(rng, m, n, k, bits, top=0, spread=1.0):
    """Inputs of one vocabulary matrix; rows of x lean towards a listed entry."""
    d = {"codes": make_codes(rng, n, k, bits), "scales": make_scales(rng, n), "bits": bits}
    d["w"] = weights(d["codes"], d["scales"], k, bits)
    width = max(top, 1)
    d["index"] = rng.integers(0, n, (m, width)).astype(np.int32)
    d["logits"] = (rng.standard_normal((m, width)) * 3).astype(np.float32)
    x = rng.standard_normal((m, k)) * spread
    lean = rng.uniform(0, 8, (m, 1)) / np.maximum(1e-9, (d["w"][d["index"][:, 0]] ** 2).sum(1, keepdims=True))
    d["x_bits"], d["x"] = bf16(x + lean * d["w"][d["index"][:, 0]])
    return d


def loss(d, index, logits=None, t=1.0):
    """{"loss", "lse", "dx"}: (value, bound) of each; logits None: cross entropy (index [m, 1], t 1)."""
    x, w = d["x"], d["w"]
    n, k = w.shape
    m = x.shape[0]
    l = x @ w.T / t
    el = (k * E24 * (np.abs(x) @ np.abs(w).T) + 3 * E24 * np.abs(x @ w.T)) / t
    r = l.max(1, keepdims=True)
    lse = r + np.log(np.exp(l - r).sum(1, keepdims=True))
    e_lse = el.max(1, keepdims=True) + 2.0 ** -17 + 4 * E24 * np.abs(lse)
    p = np.exp(l - lse)
    valid = (index >= 0) & (index < n)
    z = np.zeros(index.shape) if logits is None else logits.astype(np.float64) / t
    z = np.where(valid, z, -np.inf)
    alive = (z > -np.inf).any(1, keepdims=True)
    zr = np.where(alive, z.max(1, keepdims=True), 0)
    total = np.where(alive, np.exp(z - zr).sum(1, keepdims=True), 1)
    with np.errstate(divide="ignore", invalid="ignore"):
        log_q = np.where(z > -np.inf, z - zr - np.log(total), 0)
    q = np.where(alive & (z > -np.inf), np.exp(log_q), 0)
    at = np.where(valid, index, 0)
    l_at, el_at = np.take_along_axis(l, at, 1), np.take_along_axis(el, at, 1)
    value = (q * (log_q - l_at + lse)).sum(1)
    z_err = 3 * E24 * np.abs(np.where(q > 0, z, 0))
    q_rel = 2.0 ** -19 + 2 * z_err.max(1, keepdims=True)
    err = (q * (q_rel * (1 + np.abs(log_q) + np.abs(lse - l_at)) + 4 * E24 * np.abs(log_q) + el_at + e_lse)).sum(1)
    d_logits, d_err = p.copy(), p * (el + e_lse)
    for i in range(m):
        places = set(index[i][valid[i]].tolist())
        if len(places) == 1 and alive[i, 0]:  # one entry: relative accuracy
            # (from the others' sum here too: the difference in float64 has lost its digits where 1 - p is 1e-13)
            others = np.exp(np.delete(l[i], list(places)) - l_at[i][valid[i]][0]).sum()
            rest, log_p = others / (1 + others), -np.log1p(others)
            value[i] = (q[i] * log_q[i]).sum() - log_p
            err[i] = rest * (2 * e_lse[i, 0]) + 2.0 ** -20 * abs(log_p) + (q[i] * (q_rel[i] * (1 + np.abs(log_q[i])))).sum() * (len(index[i]) > 1)
        for j in range(index.shape[1]):
            if valid[i, j]:
                d_logits[i, index[i, j]] -= q[i, j]
                d_err[i, index[i, j]] += q[i, j] * q_rel[i, 0]
        if len(places) == 1 and alive[i, 0]:
            d_logits[i, list(places)[0]] = -rest
            d_err[i, list(places)[0]] = rest * (2 * e_lse[i, 0])
    d_err = t * (d_err + 2.0 ** -8 * (np.abs(d_logits) + d_err)) * alive
    d_err += t * 2.0 ** -8 * p * alive
    d_logits = t * d_logits * alive
    dx = d_logits @ w
    dx_err = d_err @ np.abs(w) + (n + 4) * E24 * (np.abs(d_logits) + d_err) @ np.abs(w)
    value, err = t * t * value * alive[:, 0], t * t * err * alive[:, 0]
    return {"loss": (value, err * (1 + 2.0 ** -20) + 4 * E24 * np.abs(value)), "lse": (lse[:, 0], e_lse[:, 0]),
            "dx": (dx, rounded(dx_err, dx) * alive)}


def check(name, got, want, bound):
    got = np.asarray(got, dtype=np.float64)
    off = np.abs(got - want)
    bad = ~(off <= bound)
    if bad.any():
        at = np.argwhere(bad)[0]
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} out of bounds, at {at.tolist()}: got "
                             f"{got[tuple(at)]!r}, want {want[tuple(at)]!r} within {np.broadcast_to(bound, bad.shape)[tuple(at)]!r}")


def embed_gradient(dout, tokens, first, count, scale):
    """(value, bound) of the trained rows' gradient: a float32 sum of the rows and its product with the scale."""
    out, mag, num = np.zeros((count, dout.shape[1])), np.zeros((count, dout.shape[1])), np.zeros((count, 1))
    for r, t in enumerate(tokens.tolist()):
        if first <= t < first + count:
            out[t - first] += dout[r]
            mag[t - first] += np.abs(dout[r])
            num[t - first] += 1
    return scale * out, rounded(abs(scale) * (num + 2) * E24 * mag, scale * out) * (mag > 0)
