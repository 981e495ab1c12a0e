"""cross_entropy(), distill() and loss_backward() on the GPU against float64
(tests/vocabulary_reference.py), on both product paths."""
import numpy as np
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests import vocabulary_reference as ref
from tests.helpers import from_dev_bf16, to_dev_bf16, to_dev_codes
from workloads import bf16_bits_to_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tp.load_library()


@pytest.fixture(params=[(None, 0), (False, 0), (True, 0), (True, 4096)], ids=["auto", "few", "many", "operands"])
def path(request):
    """The library's choice, decoding in the few rows' products, the many rows' products (the first one decoding on
    its way where that is reckoned to pay), and those with all weights decoded beforehand."""
    tp.force_path(*request.param)
    yield request.param
    tp.force_path(None)


def dev(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def packed(d):
    return to_dev_codes(d["codes"]), to_dev_bf16(d["scales"]), d["bits"]


def values(t):
    return bf16_bits_to_f32(from_dev_bf16(t)).astype(np.float64)


def check_all(what, got, want):
    ref.check(what + " loss", got[0].cpu().numpy(), *want["loss"])
    ref.check(what + " lse", got[1].cpu().numpy(), *want["lse"])
    if len(got) > 2:
        ref.check(what + " dx", values(got[2]), *want["dx"])


# odd and ragged sizes: one row, one row past a tile, one vocabulary row group, a vocabulary past a tile and a span
SIZES = [(1, 4, 256, 2), (3, 20004, 256, 4), (1, 1000, 512, 4), (5, 256, 512, 2), (17, 260, 256, 3), (33, 36, 768, 4), (64, 4100, 256, 3),
         (97, 516, 512, 4), (130, 1028, 256, 2), (257, 772, 256, 4), (300, 68, 512, 3)]


@pytest.mark.parametrize("m,n,k,bits", SIZES)
def test_cross_entropy(path, m, n, k, bits):
    print(f"cross_entropy {m} {n} {k} {bits} {path}", flush=True)
    d = ref.draw(np.random.default_rng(m * 7 + n), m, n, k, bits)
    target = d["index"][:, 0].copy()
    target[::5] = [-1, n, 2**31 - 1, -2**31][m % 4]
    want = ref.loss(d, target[:, None])
    x = to_dev_bf16(d["x_bits"])
    check_all("keep", tp.cross_entropy(x, *packed(d), dev(target), keep=True), want)
    check_all("forward", tp.cross_entropy(x, *packed(d), dev(target)), want)


@pytest.mark.parametrize("top,t", [(1, 1.0), (3, 2.0), (5, 0.01), (64, 0.5), (65, 1.0), (256, 100.0)])
@pytest.mark.parametrize("m,n,k,bits", [SIZES[1], SIZES[2], SIZES[4], SIZES[5], SIZES[7], SIZES[9]])
def test_distill(path, m, n, k, bits, top, t):
    print(f"distill {m} {n} {k} {bits} top {top} T {t} {path}", flush=True)
    rng = np.random.default_rng(m * 11 + top)
    d = ref.draw(rng, m, n, k, bits, top)  # (indices repeat where the list is long)
    index, logits = d["index"].copy(), d["logits"].copy()
    out = rng.random((m, top)) < 0.2
    index[out] = rng.choice([-1, n, 2**31 - 1, -2**31], out.sum())
    logits[out] = rng.choice([np.nan, np.inf, -np.inf, 0.0, 3e38], out.sum())
    logits[rng.random((m, top)) < 0.1] = -np.inf
    if m > 2:
        index[0], logits[1] = -1, -np.inf  # rows without an entry
        index[2, 1:] = -7                  # a row with at most one
    hidden = (index < 0) | (index >= n)
    clean = np.where(hidden, 0, logits).astype(np.float32)
    want = ref.loss(d, index, clean, t)
    x = to_dev_bf16(d["x_bits"])
    got = tp.distill(x, *packed(d), dev(index), dev(logits), temperature=t, keep=True)
    check_all("keep", got, want)
    two = tp.distill(x, *packed(d), dev(index), dev(logits), temperature=t)
    check_all("forward", two, want)
    if m > 2:
        assert float(got[0][0]) == 0 and float(got[0][1]) == 0 and not got[2][:2].any()


def test_distill_of_one_entry_is_cross_entropy():
    import torch

    print("distill of one entry", flush=True)
    d = ref.draw(np.random.default_rng(3), 19, 260, 512, 4)
    x, target = to_dev_bf16(d["x_bits"]), dev(d["index"])
    a = tp.cross_entropy(x, *packed(d), target[:, 0].contiguous(), keep=True)
    b = tp.distill(x, *packed(d), target, torch.randn(19, 1, device="cuda"), keep=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("m", [3, 300])
def test_certain_targets_keep_their_digits(path, m):
    """1 - p far below float32's step at 1: loss and gradient come from the other entries' sum."""
    print(f"certain targets {m} {path}", flush=True)
    rng = np.random.default_rng(8)
    d = ref.draw(rng, m, 64, 512, 4)
    w = d["w"][d["index"][:, 0]]
    lean = np.linspace(5, 60, m)[:, None]
    d["x_bits"], d["x"] = ref.bf16(0.1 * rng.standard_normal((m, 512)) + lean * w / (w ** 2).sum(1, keepdims=True))
    want = ref.loss(d, d["index"])
    got = tp.cross_entropy(to_dev_bf16(d["x_bits"]), *packed(d), dev(d["index"][:, 0]), keep=True)
    check_all("certain", got, want)
    small = want["loss"][0] < 1e-8
    assert small.any()
    l = d["x"] @ d["w"].T
    other = np.exp(l - np.take_along_axis(l, d["index"], 1))
    np.put_along_axis(other, d["index"], 0, 1)
    np.testing.assert_allclose(got[0].cpu().numpy()[small], np.log1p(other.sum(1))[small], rtol=1e-4)


def test_wide_logits(path):
    """Logits of hundreds, of either sign, and a likeliest entry far from the others."""
    print(f"wide logits {path}", flush=True)
    rng = np.random.default_rng(9)
    d = ref.draw(rng, 40, 516, 512, 3, spread=300.0)
    check_all("wide", tp.cross_entropy(to_dev_bf16(d["x_bits"]), *packed(d), dev(d["index"][:, 0]), keep=True),
              ref.loss(d, d["index"]))


def test_rows_do_not_meet(path):
    """An infinity or NaN in one row of x stays in it; zeros are an even distribution."""
    import torch

    print(f"rows apart {path}", flush=True)
    d = ref.draw(np.random.default_rng(10), 40, 516, 256, 4)
    x, target = to_dev_bf16(d["x_bits"]), dev(d["index"][:, 0])
    clean = tp.cross_entropy(x, *packed(d), target, keep=True)
    x[7, 3], x[20, 100], x[30] = float("inf"), float("nan"), 0
    got = tp.cross_entropy(x, *packed(d), target, keep=True)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[7, 20, 30]] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, clean))
    assert got[0][20].isnan() and got[1][20].isnan() and not got[0][7].isfinite()
    assert abs(float(got[0][30]) - np.log(516)) < 1e-5


def test_a_teacher_that_is_not_a_number(path):
    """A NaN or infinite logit of a valid entry reaches its row alone."""
    import torch

    print(f"teacher NaN {path}", flush=True)
    d = ref.draw(np.random.default_rng(14), 40, 516, 256, 4, top=4)
    x, index, z = to_dev_bf16(d["x_bits"]), dev(d["index"]), dev(d["logits"])
    clean = tp.distill(x, *packed(d), index, z, keep=True)
    z[3, 1], z[11, 2] = float("nan"), float("inf")
    x[20, 7] = float("inf")
    got = tp.distill(x, *packed(d), index, z, keep=True)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[3, 11, 20]] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, clean))
    assert got[0][[3, 11]].isnan().all() and torch.equal(got[1][[3, 11]], clean[1][[3, 11]])
    assert got[2][3].isnan().any() and not got[0][20].isfinite()


def test_several_slabs_and_chunks():
    """Weights decoded a few tiles at a time."""
    print("slabs", flush=True)
    d = ref.draw(np.random.default_rng(11), 150, 2052, 512, 4, top=5)
    want = ref.loss(d, d["index"], d["logits"], 1.5)
    try:
        tp.force_path(True, 16)
        got = tp.distill(to_dev_bf16(d["x_bits"]), *packed(d), dev(d["index"]), dev(d["logits"]), temperature=1.5,
                         keep=True)
    finally:
        tp.force_path(None)
    check_all("slabs", got, want)


def test_gradient_against_differences():
    """The loss along dx: (loss(x + h v) - loss(x - h v)) / 2h over the rows, in the float64 formula and in the
    library's own losses. Bounds: the losses' own errors over 2h, and the third derivative's h^2 |v w|^3."""
    print("differences", flush=True)
    rng = np.random.default_rng(12)
    d = ref.draw(rng, 9, 132, 256, 4, top=4)
    x = to_dev_bf16(d["x_bits"])
    lists = dev(d["index"]), dev(d["logits"])
    dx = values(tp.distill(x, *packed(d), *lists, temperature=1.3, keep=True)[2])
    v = np.sign(dx) * 0.25  # (x + v is rounded to bf16: the step is the rounded one)
    up, down = ref.bf16(d["x"] + v), ref.bf16(d["x"] - v)
    step = up[1] - down[1]
    got = [tp.distill(to_dev_bf16(b), *packed(d), *lists, temperature=1.3)[0].cpu().numpy().astype(np.float64)
           for b in (up[0], down[0])]
    errs = [ref.loss(dict(d, x=u), d["index"], d["logits"], 1.3)["loss"][1] for u in (up[1], down[1])]
    want = ref.loss(d, d["index"], d["logits"], 1.3)
    # second-order and higher terms, exactly, from the float64 losses
    exact = [ref.loss(dict(d, x=u), d["index"], d["logits"], 1.3)["loss"][0] for u in (up[1], down[1])]
    curve = (exact[0] - exact[1]) - (want["dx"][0] * step).sum(1)
    bound = errs[0] + errs[1] + (want["dx"][1] * np.abs(step)).sum(1) + 1e-9
    ref.check("along dx", got[0] - got[1] - curve, (dx * step).sum(1), bound)
    assert (np.abs(exact[0] - exact[1]) > 20 * np.abs(curve)).any()  # the differences say something


def test_loss_backward():
    import torch

    print("loss_backward", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    dx = torch.randn(37, 768, generator=g, device="cuda").bfloat16()
    f = torch.randn(37, generator=g, device="cuda")
    want = (dx.float() * f[:, None]).bfloat16()
    assert torch.equal(tp.loss_backward(f, dx), want)
    own = dx.clone()
    assert tp.loss_backward(f, own, out=own) is own and torch.equal(own, want)
    with pytest.raises(ValueError):
        tp.loss_backward(f, dx[:, :255].contiguous())


def test_refusals():
    import torch

    print("refusals", flush=True)
    d = ref.draw(np.random.default_rng(13), 3, 36, 256, 4, top=2)
    x, target, index, logits = (to_dev_bf16(d["x_bits"]), dev(d["index"][:, 0].copy()), dev(d["index"]),
                                dev(d["logits"]))
    p = packed(d)
    for bad in (target.long(), target[:2], target[:, None], target.cpu()):
        with pytest.raises((TypeError, ValueError)):
            tp.cross_entropy(x, *p, bad)
    for bad_i, bad_z in ((index.long(), logits), (index, logits.double()), (index[:, :1], logits), (index, logits[:2]),
                         (index[:, 0], logits), (index[:, :0], logits[:, :0]), (index.t(), logits.t())):
        with pytest.raises((TypeError, ValueError)):
            tp.distill(x, *p, bad_i, bad_z)
    for t in (0.0, -1.0, 0.009, 101.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            tp.distill(x, *p, index, logits, temperature=t)
    wide = torch.zeros((3, 257), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        tp.distill(x, *p, wide, wide.float())
    with pytest.raises(ValueError):
        tp.cross_entropy(x[:0], *p, target[:0])
    with pytest.raises((TypeError, ValueError)):
        tp.cross_entropy(x.float(), *p, target)
