"""Float64 reference of the fine-tuned layers (adapters, gated block and their
gradients) on small shapes, with a bound on each output (test infrastructure).

The weights are the CPU oracle's (exact bf16 numbers); everything else is
float64 NumPy from the formulas.

Bounds. A float32 sum of L products of bf16 numbers (each product exact in
float32) is off by at most L * 2^-24 * sum|terms| in any order; products of
values that carry an error pass it on. A value that enters a matrix product as
the sum of two bf16 numbers is off by at most 2^-16 (half a step of 2^-7,
twice). The last rounding adds 2^-8 of the rounded value (half a bf16 step).
"""
from __future__ import annotations

import numpy as np

import oracle
from workloads import bf16_bits_to_f32, f32_to_bf16_bits, make_codes, make_scales

E24 = 2.0 ** -24


def weights(codes, scales, k, bits):
    return bf16_bits_to_f32(oracle.decode(codes, scales, k, bits)).astype(np.float64)


def bf16(a):
    """Values rounded to bf16, as (bit patterns, float64)."""
    bits = f32_to_bf16_bits(np.asarray(a, dtype=np.float32))
    return bits, bf16_bits_to_f32(bits).astype(np.float64)


def rounded(err, y):
    """The bound after the last rounding to bf16 (2^-133: the least subnormal's half step)."""
    return err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y) + 2.0 ** -133


def product(p, w):
    """p @ w.T with its error bound."""
    a = np.abs(p) @ np.abs(w).T
    return p @ w.T, p.shape[1] * E24 * a


def draw(rng, m, n, k, bits, rank=0, count=0):
    """Inputs of one layer; with a rank, an adapter set."""
    d = {"codes": make_codes(rng, n, k, bits), "scales": make_scales(rng, n)}
    d["w"] = weights(d["codes"], d["scales"], k, bits)
    d["x_bits"], d["x"] = bf16(rng.standard_normal((m, k)))
    d["dout_bits"], d["dout"] = bf16(rng.standard_normal((m, n)))
    if rank:
        d["a_bits"], d["a"] = bf16(rng.standard_normal((count, rank, k)) * k ** -0.5)
        d["b_bits"], d["b"] = bf16(rng.standard_normal((count, n, rank)) * 0.3)
        d["gain"] = rng.uniform(0.5, 2.0, count).astype(np.float32)
        d["index"] = rng.integers(-1, count, m).astype(np.int32)
    return d


def low_rank(p, f, gain, index):
    """v[m] = gain F[i] p[m], F [count, rank, C]; float64 with its bound."""
    m, rank = p.shape[0], f.shape[1]
    v, e = np.zeros((m, rank)), np.zeros((m, rank))
    for i in range(f.shape[0]):
        of = np.nonzero(index == i)[0]
        y, err = product(p[of], f[i])
        v[of] = gain[i] * y
        e[of] = gain[i] * err + E24 * np.abs(v[of]) + (gain[i] * err) * E24
    return v, e


def spread(v, e, f, index, width):
    """sum_r F[i][c][r] v[m, r], F [count, C, rank], with its bound."""
    y, err = np.zeros((v.shape[0], width)), np.zeros((v.shape[0], width))
    for i in range(f.shape[0]):
        of = np.nonzero(index == i)[0]
        y[of] = v[of] @ f[i].T
        mag = np.abs(v[of]) @ np.abs(f[i]).T
        err[of] = e[of] @ np.abs(f[i]).T + (2.0 ** -16 + 2 * (v.shape[1] + 32) * E24) * mag
    return y, err


def adapters(d):
    """out and its bound."""
    y, e = product(d["x"], d["w"])
    t, te = low_rank(d["x"], d["a"], d["gain"].astype(np.float64), d["index"])
    z, ze = spread(t, te, d["b"], d["index"], d["w"].shape[0])
    out = y + z
    return out, rounded(e + ze + 4 * E24 * (np.abs(y) + np.abs(z)), out)


def adapters_backward(d):
    """{dx, da, db}: (value, bound)."""
    gain, index = d["gain"].astype(np.float64), d["index"]
    y, e = product(d["dout"], d["w"].T)
    u, ue = low_rank(d["dout"], d["b"].transpose(0, 2, 1), gain, index)
    t, te = low_rank(d["x"], d["a"], gain, index)
    z, ze = spread(u, ue, d["a"].transpose(0, 2, 1), index, d["x"].shape[1])
    dx = y + z
    da, db, dae, dbe = np.zeros_like(d["a"]), np.zeros_like(d["b"]), np.zeros_like(d["a"]), np.zeros_like(d["b"])
    for i in range(d["a"].shape[0]):
        of = np.nonzero(index == i)[0]
        share = 2.0 ** -16 + 2 * (d["x"].shape[0] + 32) * E24
        da[i], db[i] = u[of].T @ d["x"][of], d["dout"][of].T @ t[of]
        dae[i] = (ue[of] + share * np.abs(u[of])).T @ np.abs(d["x"][of])
        dbe[i] = np.abs(d["dout"][of]).T @ (te[of] + share * np.abs(t[of]))
    return {"dx": (dx, rounded(e + ze + 4 * E24 * (np.abs(y) + np.abs(z)), dx)),
            "da": (da, rounded(dae, da)), "db": (db, rounded(dbe, db))}


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def gated(x, wg, wu):
    """{h, gate, up}: (value, bound). |silu'| <= 1.1; the float32 evaluation of
    silu(gate) * up is off by at most 2^-20 of it (exp within 2 steps of its
    value plus 2^-24 |gate| from its argument, four more operations; |gate| < 8
    where silu(gate) is not negligible against its own bound)."""
    g, ge = product(x, wg)
    u, ue = product(x, wu)
    silu = g * sigmoid(g)
    h = silu * u
    he = 1.1 * ge * (np.abs(u) + ue) + np.abs(silu) * ue + (2.0 ** -20 + np.abs(g) * 2.0 ** -22) * np.abs(h)
    return {"h": (h, rounded(he, h)), "gate": (g, rounded(ge, g)), "up": (u, rounded(ue, u))}


def gated_grads(dh, gate, up):
    """{dgate, dup}: (value, bound) of the elementwise part."""
    s = sigmoid(gate)
    dup, dgate = dh * gate * s, dh * up * s * (1 + gate * (1 - s))
    rel = 2.0 ** -20 + np.abs(gate) * 2.0 ** -22
    mag = np.abs(dh * up * s) * (1 + np.abs(gate) * (1 - s))
    return {"dgate": (dgate, rounded(rel * mag + np.abs(dh * up * s * gate) * 2.0 ** -22, dgate)),
            "dup": (dup, rounded(rel * np.abs(dup), dup))}


def check(name, got_bits, value, bound):
    """Every output within its bound, NaN and infinities at the same places."""
    got = bf16_bits_to_f32(got_bits).astype(np.float64)
    assert got.shape == value.shape, f"{name}: {got.shape} against {value.shape}"
    fine = np.isfinite(value)
    assert np.array_equal(np.isnan(got), np.isnan(value)), f"{name}: NaN at other places"
    off = np.abs(got - value)
    bad = fine & ~(off <= bound)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} out of bound, first at {at}: "
                             f"{got[at]!r} against {value[at]!r}, bound {bound[at]!r}")
