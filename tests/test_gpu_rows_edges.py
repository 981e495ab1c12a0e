"""The fine-tuned layers at the edges of what the header allows: operands at the
least alignment, low-rank sums over many spans, gated_backward where element
offsets pass 32 bits, and contractions so long that the decoded weights go in
several launches.

Bounds are those of tests/rows_reference.py, except for sums of tens of
thousands of terms, where the worst case (L 2^-24 of the terms' magnitudes) would
hide a wrong term: L roundings of partial sums of up to 4 sqrt(L) s, s the terms'
size, whose signs vary, come to 4 L s 2^-24 (with L s^2 the sum of the terms'
squares), and the result is rounded to bf16 (2^-8 of it).
"""
import numpy as np
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests import rows_reference as ref
from tests.helpers import from_dev_bf16, to_dev_bf16, to_dev_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tp.load_library()
    yield
    torch.cuda.empty_cache()


@pytest.fixture
def force_path():
    """Setter for the library's product path; its own choice is restored when the test ends."""
    yield tp.force_path
    tp.force_path(None)


def on_gpu(d):
    import torch

    return dict(x=to_dev_bf16(d["x_bits"]), codes=to_dev_codes(d["codes"]), scales=to_dev_bf16(d["scales"]),
                a=to_dev_bf16(d["a_bits"]), b=to_dev_bf16(d["b_bits"]), gain=torch.from_numpy(d["gain"]).cuda(),
                index=torch.from_numpy(d["index"]).cuda()), to_dev_bf16(d["dout_bits"])


def moved(t, by):
    """A copy that starts `by` bytes past a 256-byte boundary."""
    import torch

    step = by // t.element_size()
    room = torch.empty(t.numel() + step, dtype=t.dtype, device=t.device)
    assert room.data_ptr() % 256 == 0 and by % t.element_size() == 0
    out = room[step:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("bits", [2, 3, 4])
def test_operands_at_their_least_alignment(force_path, bits, path):
    import torch

    print(f"edges alignment bits={bits} path={path}", flush=True)
    m, n, k = 37, 132, 512
    d = ref.draw(np.random.default_rng(70 + bits), m, n, k, bits, rank=5, count=3)
    s, dout = on_gpu(d)
    gate, up = tp.gated(s["x"], s["codes"], s["scales"], s["codes"], s["scales"], bits, keep=True)[1:]
    force_path(path)

    def calls(at):
        q = {name: at(t) for name, t in s.items()}
        g = at(dout)
        x, packed = q["x"], (q["codes"], q["scales"], q["codes"], q["scales"], bits)
        like = lambda t: at(torch.zeros_like(t))
        return [tp.adapters(bits=bits, out=like(dout), **q),
                *tp.adapters_backward(g, bits=bits, dx=like(x), da=like(q["a"]), db=like(q["b"]), **q),
                tp.gated(x, *packed, out=like(dout)),
                *tp.gated_backward(g, at(gate), at(up), *packed, dx=like(x), dgate=like(dout), dup=like(dout))]

    least = {id(s["scales"]): 2, id(s["gain"]): 4, id(s["index"]): 4}
    aligned = calls(lambda t: t)
    for got, want in zip(calls(lambda t: moved(t, least.get(id(t), 16))), aligned):
        assert torch.equal(got, want)


# The forward sums run over K and the backward's over N: 17408 columns give
# each of up to 128 rows more spans than a thread adds in one batch (16).
@pytest.mark.parametrize("n,k", [(36, 17408), (17408, 256)])
@pytest.mark.parametrize("m,count", [(1, 1), (20, 9), (97, 3)])
def test_low_rank_sums_of_many_spans(m, count, n, k):
    print(f"edges spans m={m} n={n} k={k}", flush=True)
    d = ref.draw(np.random.default_rng(80 + m + n), m, n, k, 2, rank=33, count=count)
    d["index"][0] = 0
    s, dout = on_gpu(d)
    out = tp.adapters(bits=2, **s)
    ref.check(f"spans out m={m} n={n}", from_dev_bf16(out), *ref.adapters(d))
    want = ref.adapters_backward(d)
    for name, t in zip(("dx", "da", "db"), tp.adapters_backward(dout, bits=2, **s)):
        ref.check(f"spans {name} m={m} n={n}", from_dev_bf16(t), *want[name])


def layer(g, n, k, bits):
    import torch

    codes = torch.randint(-2**31, 2**31 - 1, (n, k * bits // 32), generator=g, device="cuda", dtype=torch.int32)
    return codes, (torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005).to(torch.bfloat16)


def normal(g, *shape):
    import torch

    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return t.normal_(generator=g)


def long_sum(p, w):
    """p @ w in 64 bits with the bound of its float32 sum rounded to bf16 (see above)."""
    value = p @ w
    squares = (p * p) @ (w * w)
    return value, 4 * p.shape[1] ** 0.5 * squares.sqrt() * 2.0 ** -24 * (1 + 2.0 ** -8) + 2.0 ** -8 * value.abs()


def need_memory(gib):
    import torch

    if torch.cuda.get_device_properties(0).total_memory < gib << 30:
        pytest.skip(f"needs {gib} GiB")


def test_gated_backward_past_32_bits():
    import torch

    need_memory(96)
    m, n, k, bits = 140000, 17408, 256, 2
    assert m * n > 2**31
    print(f"edges gated_backward m={m} n={n}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(71)
    packed = (*layer(g, n, k, bits), *layer(g, n, k, bits), bits)
    wg, wu = (tp.decode(c, s, k, bits) for c, s in (packed[:2], packed[2:4]))
    rows = torch.cat([torch.arange(40), torch.arange(2**31 // n - 20, 2**31 // n + 20), torch.arange(m - 40, m)]).cuda()
    x = normal(g, m, k)
    h, gate, up = tp.gated(x, *packed, keep=True)
    want = ref.gated(x[rows].double().cpu().numpy(), wg.double().cpu().numpy(), wu.double().cpu().numpy())
    for name, t in (("h", h), ("gate", gate), ("up", up)):
        ref.check(f"large {name}", from_dev_bf16(t[rows].contiguous()), *want[name])
    del x, want
    dh = h.normal_(generator=g)
    dx, dgate, dup = tp.gated_backward(dh, gate, up, *packed)
    few = [t[rows].contiguous() for t in (dh, gate, up)]
    fx, fgate, fup = tp.gated_backward(*few, *packed)
    # elementwise, the same arithmetic whatever the number of rows
    assert torch.equal(dgate[rows], fgate) and torch.equal(dup[rows], fup)
    grads = ref.gated_grads(*(t[:8].double().cpu().numpy() for t in few))
    for name, t in (("dgate", fgate), ("dup", fup)):
        ref.check(f"large {name}", from_dev_bf16(t[:8].contiguous()), *grads[name])
    value, bound = long_sum(torch.cat([fgate, fup], 1).double(), torch.cat([wg, wu], 0).double())
    for got in (dx[rows], fx):
        assert bool(((got.double() - value).abs() <= bound).all())
    torch.cuda.synchronize()


def test_weights_of_a_long_contraction_in_several_launches(force_path):
    import torch

    need_memory(64)
    # 128 operand tiles of 9.6 MB: more than the 1 GiB of one launch
    m, n, k, bits, rank = 700, 300000, 2048, 2, 4
    print(f"edges long contraction n={n}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(72)
    codes, scales = layer(g, n, k, bits)
    w = tp.decode(codes, scales, k, bits)
    x, dout = normal(g, m, k), normal(g, m, n)
    a, b, gain = normal(g, 2, rank, k) * 0.03, normal(g, 2, n, rank) * 0.03, torch.tensor([1.0, 0.5], device="cuda")
    index = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    index[100:120] = 1
    plain = torch.cat([torch.arange(40), torch.arange(m - 40, m)]).cuda()
    value, bound = long_sum(dout[plain].double(), w.double())
    both = []
    for path in (True, False):
        force_path(path)
        dx, da, db = tp.adapters_backward(dout, x, codes, scales, bits, a, b, gain, index)
        assert bool(((dx[plain].double() - value).abs() <= bound).all())
        both.append((da, db))
        assert not bool(da[0].any()) and not bool(db[0].any()) and bool(da[1].any()) and bool(db[1].any())
    assert all(torch.equal(p, q) for p, q in zip(*both))  # the low-rank sums are the same launches
    torch.cuda.synchronize()
