"""distill()'s lists on the GPU, on all paths: logits of any float32 value."""
import numpy as np
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests import vocabulary_reference as ref
from tests.helpers import to_dev_bf16
from tests.test_gpu_loss import check_all, dev, need_gpu, packed, path  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min


def check(what, d, t, got, want):
    """check_all() with float32's range: at T = 0.01 a row's only entry is so likely that its loss and all p are below
    the smallest normal float32, 2^-126, where the hardware's exponential gives 0 and the reference's bounds, being
    relative, go on falling. An exponential is then off by up to 2^-126, and so is the loss, before the factor T^2 and
    again as a result: (1 + T^2) 2^-126. Each of N terms of dx is off by as much, times T |W|, in the exponential,
    in the operand and in the term itself: 3 N (1 + T) 2^-126 max|W|."""
    tiny = 2.0 ** -126
    floor = {"loss": (1 + t * t) * tiny, "lse": 0.0,
             "dx": 3 * len(d["w"]) * (1 + t) * tiny * max(1.0, np.abs(d["w"]).max())}
    check_all(what, got, {k: (value, bound + floor[k]) for k, (value, bound) in want.items()})


def distill(d, index, logits, t):
    return tp.distill(to_dev_bf16(d["x_bits"]), *packed(d), dev(index), dev(logits), temperature=t, keep=True)


@pytest.mark.parametrize("top,t", [(1, 1.0), (1, 0.01), (4, 1.0), (4, 0.01), (70, 2.0)])
@pytest.mark.parametrize("m,n", [(5, 260), (3, 20004), (300, 260)])
def test_teachers_of_the_largest_and_lowest_logits(path, m, n, top, t):  # noqa: F811
    """Finite logits that float32 cannot hold once they are scaled by 1 / T: only their differences count."""
    import torch

    print(f"largest logits {m} {n} top {top} T {t} {path}", flush=True)
    d = ref.draw(np.random.default_rng(m + n + top), m, n, 256, 4, top=top)
    even = distill(d, d["index"], np.zeros((m, top), np.float32), t)
    check("even", d, t, even, ref.loss(d, d["index"], np.zeros((m, top), np.float32), t))
    for z in (LOWEST, -LOWEST, np.float32(-3e36), np.float32(3e38)):
        got = distill(d, d["index"], np.full((m, top), z, np.float32), t)
        assert all(torch.equal(a, b) for a, b in zip(got, even)), z
    # an entry that a mask of the type's lowest value hides: probability 0, but not none
    logits = d["logits"].copy()
    logits[:, 1::2] = LOWEST
    check("masked", d, t, distill(d, d["index"], logits, t), ref.loss(d, d["index"], logits, t))


@pytest.mark.parametrize("top", [2, 5, 70])
@pytest.mark.parametrize("m,n,t", [(5, 260, 1.0), (3, 20004, 2.0), (300, 260, 0.5), (70, 1028, 1.0)])
def test_entries_of_no_logit_are_none(path, m, n, top, t):  # noqa: F811
    """Bit for bit what the same list gives with those entries outside the vocabulary."""
    import torch

    print(f"-inf entries {m} {n} top {top} T {t} {path}", flush=True)
    rng = np.random.default_rng(m * 3 + n + top)
    d = ref.draw(rng, m, n, 256, 4, top=top)
    index, logits = d["index"].copy(), d["logits"].copy()
    index[:, -1] = index[:, 0]  # named twice, in some rows once with a logit and once without
    gone = rng.random((m, top)) < 0.5
    gone[::3, 1:] = True        # rows of one entry, or none
    logits[gone] = -np.inf
    hidden = np.where(gone, -1, index).astype(np.int32)
    got, want = distill(d, index, logits, t), distill(d, hidden, logits, t)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    check("none", d, t, got, ref.loss(d, hidden, logits, t))


@pytest.mark.parametrize("n", [64, 20004])
@pytest.mark.parametrize("m", [3, 300])
def test_a_certain_entry_beside_entries_of_no_logit(path, m, n):  # noqa: F811
    """A list of one entry, padded with others whose logits are -inf: 1 - p and the loss far below float32's step at 1
    come from the others' sum, as in a list of that entry alone."""
    print(f"certain entry, padded list {m} {n} {path}", flush=True)
    rng = np.random.default_rng(8 + n)
    d = ref.draw(rng, m, n, 512, 4, top=4)
    d["index"] = (d["index"][:, :1] + np.array([0, 1, 7, 0])) % n  # the last names the first again
    w = d["w"][d["index"][:, 0]]
    lean = np.linspace(15, 60, m)[:, None]
    d["x_bits"], d["x"] = ref.bf16(0.1 * rng.standard_normal((m, 512)) + lean * w / (w ** 2).sum(1, keepdims=True))
    logits = np.full((m, 4), -np.inf, np.float32)
    logits[:, 0] = rng.standard_normal(m)
    logits[::2, 3] = 0.5
    got = distill(d, d["index"].astype(np.int32), logits, 1.0)
    want = ref.loss(d, np.where(logits > -np.inf, d["index"], -1), logits, 1.0)
    check("padded", d, 1.0, got, want)
    alone = np.arange(m) % 2 == 1  # (an entry named twice has its q in two parts, whose logarithms are off by 2^-24)
    small = alone & (want["loss"][0] < 1e-8)
    assert small.any()
    np.testing.assert_allclose(got[0].cpu().numpy()[small], want["loss"][0][small], rtol=1e-4)


@pytest.mark.parametrize("forced,chunk", [((False, 0), 256), ((True, 0), 512)], ids=["few", "many"])
def test_lists_over_several_chunks_of_rows(forced, chunk):
    """A vocabulary of 2^20 entries takes 256 or 512 rows at a time: ragged lists of every chunk, the last one short,
    against the formula in float64 on the GPU, and the first chunk's rows as a call of their own. Bounds as in
    test_chunks_of_rows (tests/test_gpu_vocabulary_run.py), in units of T; q is off by 2^-18 of itself."""
    import torch

    print(f"chunks of lists {forced}", flush=True)
    m, n, k, bits, top, t = 600, 1 << 20, 256, 2, 7, 1.5
    g = torch.Generator(device="cuda").manual_seed(21)
    codes = torch.randint(-2**31, 2**31, (n, k * bits // 32), generator=g, device="cuda", dtype=torch.int32)
    scales = (torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005).bfloat16()
    x = (torch.randn(m, k, generator=g, device="cuda") * 4).bfloat16()
    index = torch.randint(0, n, (m, top), generator=g, device="cuda", dtype=torch.int32)
    logits = torch.randn(m, top, generator=g, device="cuda") * 3
    length = torch.randint(0, top + 1, (m, 1), generator=g, device="cuda")
    index.masked_fill_(torch.arange(top, device="cuda") >= length, -1)  # lists of none to all
    logits[::5, 1] = -float("inf")
    try:
        tp.force_path(*forced)
        got = tp.distill(x, codes, scales, bits, index, logits, temperature=t, keep=True)
        short = tp.distill(x, codes, scales, bits, index, logits, temperature=t)
        first = tp.distill(x[:chunk], codes, scales, bits, index[:chunk], logits[:chunk], temperature=t, keep=True)
    finally:
        tp.force_path(None)
    assert all(torch.equal(a[:chunk], b) for a, b in zip(got, first))
    e24 = 2.0 ** -24
    w = tp.decode(codes, scales, k, bits).double()
    largest = w.abs().max()
    for r0 in range(0, m, 100):
        r = slice(r0, r0 + 100)
        l = x[r].double() @ w.T / t
        lse = torch.logsumexp(l, 1, keepdim=True)
        there = (index[r] >= 0) & (logits[r] > -float("inf"))
        z = torch.where(there, logits[r].double() / t, -float("inf"))
        some = there.any(1, keepdim=True)
        q = torch.where(some, torch.softmax(torch.where(some, z, 0.0), 1), 0.0)
        log_q = torch.where(q > 0, q, 1.0).log()
        at = index[r].clamp(0).long()
        off = torch.where(q > 0, lse - l.gather(1, at), 0.0)
        loss = t * t * (q * (log_q + off)).sum(1)
        d = (l - lse).exp_() * some
        d.scatter_add_(1, at, -q)
        dx = t * (d @ w)
        el = (k * e24 * (x[r].double().abs().sum(1) * largest) + 4 * e24 * 40) / t
        bound = 2 * el + 2.0 ** -17 + 8 * e24 * lse[:, 0].abs()
        worst = 2 * bound + 2.0 ** -18 * (1 + log_q.abs().amax(1) + off.abs().amax(1))
        for o in (got, short):
            assert ((o[0][r] - loss).abs() <= t * t * worst).all() and ((o[1][r] - lse[:, 0]).abs() <= bound).all()
        err = (got[2][r].double() - dx).abs()
        assert (err <= t * 2 * largest * (2 * 2.0 ** -8 + 2 * bound[:, None]) + 2.0 ** -8 * dx.abs()).all()
        assert (err.norm(dim=1) <= 2.0 ** -7 * dx.norm(dim=1) + 1e-6).all()
        assert not got[2][r][~some[:, 0]].any() and not got[0][r][~some[:, 0]].any()
