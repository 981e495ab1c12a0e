"""embed() and embed_backward() on the GPU: the lookup bit for bit against the
CPU oracle's weights, the gradient against float64."""
import numpy as np
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests import vocabulary_reference as ref
from tests.helpers import from_dev_bf16, to_dev_bf16, to_dev_codes
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tp.load_library()


def dev(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("m,n,k,count,scale", [(1, 4, 256, 0, 1.0), (7, 260, 512, 3, 22.627417), (300, 36, 768, 40, -0.3),
                                               (65, 1000, 1280, 1, 0.0)])
def test_embed(m, n, k, count, scale, bits):
    print(f"embed {m} {n} {k} {count} {bits}", flush=True)
    rng = np.random.default_rng(m + bits)
    d = ref.draw(rng, 1, n, k, bits)
    d["scales"][rng.integers(0, n, 3)] = f32_to_bf16_bits(np.float32([2.0 ** -120, -0.01, 2.0 ** 115]))
    w = ref.weights(d["codes"], d["scales"], k, bits)
    extra_bits, extra = ref.bf16(rng.standard_normal((count, k)))
    tokens = rng.integers(0, n + count, m).astype(np.int32)
    tokens[rng.random(m) < 0.2] = -1
    if m > 7:
        tokens[:4] = [n + count, 2**31 - 1, -2**31, n - 1]
    rows = np.concatenate([w, extra, np.zeros((1, k))])[np.where((tokens < 0) | (tokens >= n + count), n + count, tokens)]
    want = f32_to_bf16_bits(rows.astype(np.float32) * np.float32(scale))
    got = from_dev_bf16(tp.embed(dev(tokens), to_dev_codes(d["codes"]), to_dev_bf16(d["scales"]), k, bits, scale,
                                 to_dev_bf16(extra_bits) if count else None))
    # (a weight of code 0 has either sign)
    assert np.array_equal(bf16_bits_to_f32(got), bf16_bits_to_f32(want))


# pairs of one, two and three bytes; one workgroup of the sort and several; runs
# within a chunk, over chunk borders and over all of them
GRADIENTS = [(1, 256, 1, "any"), (7, 256, 3, "any"), (300, 512, 40, "any"), (300, 256, 1000, "none"), (2500, 256, 1, "same"),
             (5000, 768, 300, "skewed"), (5000, 256, 70000, "any"), (20000, 256, 5, "any"), (33000, 256, 2000, "skewed"), (16384, 256, 70000, "skewed"),
             (16385, 512, 300, "same"),
             (4096, 1280, 256, "sorted")]


def gradient_tokens(rng, m, first, count, kind):
    if kind == "none":
        return rng.integers(0, first, m).astype(np.int32)
    if kind == "same":
        return np.full(m, first, np.int32)
    if kind == "sorted":
        return (first + np.sort(rng.integers(0, count, m))).astype(np.int32)
    tokens = rng.integers(first - 5, first + count + 5, m)
    if kind == "skewed":
        tokens = first + np.minimum(count - 1, (rng.pareto(0.7, m) * 2).astype(np.int64))
    tokens[rng.random(m) < 0.1] = rng.choice([-1, -2**31, 2**31 - 1, first - 1])
    return tokens.astype(np.int32)


@pytest.mark.parametrize("m,k,count,kind", GRADIENTS)
def test_embed_backward(m, k, count, kind):
    import torch

    print(f"embed_backward {m} {k} {count} {kind}", flush=True)
    rng = np.random.default_rng(m + count)
    first, scale = 1000, 1.7
    tokens = gradient_tokens(rng, m, first, count, kind)
    bits, dout = ref.bf16(rng.standard_normal((m, k)))
    out = torch.full((count, k), float("nan"), dtype=torch.bfloat16, device="cuda")
    args = to_dev_bf16(bits), dev(tokens), first, count, scale
    got = tp.embed_backward(*args, dextra=out)
    value, bound = ref.embed_gradient(dout, tokens, first, count, float(np.float32(scale)))
    ref.check("dextra", bf16_bits_to_f32(from_dev_bf16(got)), value, bound)
    for _ in range(3):
        assert torch.equal(tp.embed_backward(*args), got)


@pytest.mark.parametrize("m,count,kind", [(1024, 257, "any"), (1025, 257, "any"), (16384, 257, "skewed"), (1025, 16384, "sorted"),
                                          (16384, 16385, "any"), (16384, 20000, "same"), (9000, 4097, "skewed"), (2047, 63 * 256 + 1, "none")])
def test_gradient_of_rows_sorted_by_several_workgroups(m, count, kind):
    test_embed_backward(m, 256, count, kind)


# runs of 16-row chunks that begin and end inside and at the borders of 32 neighbouring chunks
@pytest.mark.parametrize("m,runs", [(16384, [16384]), (16384, [512, 512, 15360]), (16384, [500, 40, 600, 4, 8192, 7000, 48]), (600, [30, 514, 56]),
                                    (1040, [16, 1024]), (1056, [16, 1040]), (1024, [1008, 16]), (1040, [511, 2, 511, 16]), (40000, [9, 20000, 19000, 991])])
@pytest.mark.parametrize("k", [256, 1280])
def test_gradient_of_long_runs(m, runs, k):
    import torch

    print(f"embed_backward {m} {runs} {k}", flush=True)
    rng = np.random.default_rng(m + len(runs))
    tokens = np.repeat(np.arange(len(runs), dtype=np.int32), runs)
    bits, dout = ref.bf16(rng.standard_normal((m, k)))
    args = to_dev_bf16(bits), dev(tokens), 0, len(runs) + 1
    got = tp.embed_backward(*args)
    value, bound = ref.embed_gradient(dout, tokens, 0, len(runs) + 1, 1.0)
    ref.check("dextra", bf16_bits_to_f32(from_dev_bf16(got)), value, bound)
    for _ in range(3):
        assert torch.equal(tp.embed_backward(*args), got)


@pytest.mark.parametrize("m", [1024, 1025, 16384, 16385])
@pytest.mark.parametrize("count", [2**18, 2**18 + 1, 2**22])
def test_gradient_of_the_most_trained_rows(m, count):
    """Each token once: its row is dout's, all others are zero."""
    import torch

    print(f"embed_backward {m} rows of {count}", flush=True)
    rng = np.random.default_rng(m + count)
    tokens = rng.choice(count, m, replace=False)
    tokens[:2] = [0, count - 1] if not np.isin([0, count - 1], tokens[2:]).any() else tokens[:2]
    dout = torch.randn(m, 256, device="cuda").bfloat16()
    at = torch.from_numpy(tokens).cuda()
    want = torch.zeros(count, 256, dtype=torch.bfloat16, device="cuda")
    want[at] = dout
    got = tp.embed_backward(dout, (at + 77).int(), 77, count, dextra=torch.full_like(want, float("nan")))
    assert torch.equal(got, want)


def test_one_token_everywhere_and_infinities():
    """An infinity reaches its token's row alone; a rows' order decides nothing but the last digits."""
    import torch

    print("embed_backward infinities", flush=True)
    dout = torch.randn(100, 256, device="cuda").bfloat16()
    tokens = torch.arange(100, dtype=torch.int32, device="cuda") % 7
    clean = tp.embed_backward(dout, tokens, 0, 7)
    dout[3, 5], dout[4] = float("inf"), float("nan")
    got = tp.embed_backward(dout, tokens, 0, 7)
    assert torch.isinf(got[3, 5]) and got[4].isnan().all()
    keep = torch.tensor([0, 1, 2, 5, 6], device="cuda")
    assert torch.equal(got[keep], clean[keep])


def test_refusals():
    import torch

    print("refusals", flush=True)
    d = ref.draw(np.random.default_rng(1), 1, 36, 256, 4)
    c, s = to_dev_codes(d["codes"]), to_dev_bf16(d["scales"])
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    extra = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
    for bad in (t.long(), t[:, None], t.cpu(), t[:0]):
        with pytest.raises((TypeError, ValueError)):
            tp.embed(bad, c, s, 256, 4)
    for kw in (dict(k=128), dict(k=512), dict(extra=extra[:, :128]), dict(extra=extra.float()), dict(extra=extra[0]),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(out=extra)):
        with pytest.raises((TypeError, ValueError)):
            tp.embed(**{**dict(tokens=t, codes=c, scales=s, k=256, bits=4), **kw})
    dout = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    for args in ((dout, t, 36, 0), (dout, t, -1, 2), (dout, t, (1 << 22) + 1, 2), (dout[:2], t, 36, 2),
                 (dout, t.long(), 36, 2), (dout[:, :128].contiguous(), t, 36, 2), (dout, t, 36, (1 << 22) + 1)):
        with pytest.raises((TypeError, ValueError)):
            tp.embed_backward(*args)
    with pytest.raises(ValueError):
        tp.embed_backward(dout, t, 36, 2, scale=float("inf"))
