"""adapters() and gated() under autograd on the GPU: the gradients are the
backward calls' own, bit for bit, on whatever stream the forward call ran."""
import numpy as np
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests import rows_reference as ref
from tests.helpers import to_dev_bf16, to_dev_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tp.load_library()


M, N, K, BITS, RANK, COUNT = 37, 260, 512, 4, 8, 3


@pytest.fixture
def sets():
    """A gated block [K -> N] and a projection of its own width with adapters, as arguments of the calls."""
    import torch

    rng = np.random.default_rng(61)
    d, e = ref.draw(rng, M, N, K, BITS, rank=RANK, count=COUNT), ref.draw(rng, M, N, K, BITS)
    s = dict(x=to_dev_bf16(d["x_bits"]), codes=to_dev_codes(d["codes"]), scales=to_dev_bf16(d["scales"]), bits=BITS,
             a=to_dev_bf16(d["a_bits"]), b=to_dev_bf16(d["b_bits"]), gain=torch.from_numpy(d["gain"]).cuda(),
             index=torch.from_numpy(d["index"]).cuda())
    packed = (s["codes"], s["scales"], to_dev_codes(e["codes"]), to_dev_bf16(e["scales"]), BITS)
    return s, packed, to_dev_bf16(d["dout_bits"])


def leaf(t):
    return t.clone().requires_grad_()


def test_adapters(sets):
    import torch

    print("autograd adapters", flush=True)
    s, _, dout = sets
    want = tp.adapters_backward(dout, **s)
    leaves = {name: leaf(s[name]) for name in ("x", "a", "b")}
    out = tp.adapters(**{**s, **leaves})
    assert torch.equal(out, tp.adapters(**s))
    out.backward(dout)
    assert all(torch.equal(leaves[name].grad, w) for name, w in zip(("x", "a", "b"), want))
    # one leaf alone, and the expanded gradient of a sum
    a = leaf(s["a"])
    tp.adapters(**{**s, "a": a}).sum().backward()
    assert torch.equal(a.grad, tp.adapters_backward(torch.ones_like(dout), **s)[1])
    # a gradient that starts between the library's alignments
    whole = torch.empty(M * N + 4, dtype=torch.bfloat16, device="cuda")
    whole[4:] = dout.flatten()
    x = leaf(s["x"])
    tp.adapters(**{**s, "x": x}).backward(whole[4:].view(M, N))
    assert torch.equal(x.grad, want[0])


@pytest.mark.parametrize("keep", [False, True])
def test_gated(sets, keep):
    import torch

    print(f"autograd gated keep={keep}", flush=True)
    s, packed, dh = sets
    x = leaf(s["x"])
    got = tp.gated(x, *packed, keep=keep)
    want = tp.gated(s["x"], *packed, keep=True)
    h = got[0] if keep else got
    assert torch.equal(h, want[0])
    h.backward(dh)
    assert torch.equal(x.grad, tp.gated_backward(dh, *want[1:], *packed)[0])
    if keep:
        h, gate, up = tp.gated(x, *packed, keep=True)
        with pytest.raises(RuntimeError, match="kept projections"):
            gate.sum().backward()


def step(s, packed, x, a, b, dy, pad):
    """The block, its output brought to the projection's width, and the projection with its adapters."""
    import torch

    h = tp.gated(x, *packed)
    y = tp.adapters(torch.nn.functional.pad(h, (0, pad)), **{**{k: s[k] for k in ("codes", "scales", "bits", "gain", "index")},
                                                             "a": a, "b": b})
    return torch.autograd.grad(y, (x, a, b), dy)


def test_a_run_of_both_on_two_streams(sets):
    import torch

    print("autograd run, streams", flush=True)
    s, packed, dy = sets
    pad = K - N
    with torch.no_grad():
        h, gate, up = tp.gated(s["x"], *packed, keep=True)
        wide = torch.nn.functional.pad(h, (0, pad)).contiguous()
        dh, da, db = tp.adapters_backward(dy, **{**s, "x": wide})
        dx = tp.gated_backward(dh[:, :N].contiguous(), gate, up, *packed)[0]
    leaves = leaf(s["x"]), leaf(s["a"]), leaf(s["b"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for stream in streams:
            with torch.cuda.stream(stream):
                got.append(step(s, packed, *leaves, dy, pad))
        torch.cuda.synchronize()
        for grads in got:
            assert all(torch.equal(p, q) for p, q in zip(grads, (dx, da, db)))


def test_the_gradient_against_differences(sets):
    # The output is linear in each of x, a and b alone: a step of one of them
    # changes <dout, out> by the step times the gradient. Both outputs are
    # rounded (2^-8 of each), the gradient too; the float32 sums of K = 512 terms
    # are off by 2^-15 of the terms' magnitudes, which are some sqrt(K) = 23 times
    # the sum (23 2^-15 < 2^-10), in two outputs and the gradient: 1.5 covers both.
    import torch

    print("autograd differences", flush=True)
    s, _, dout = sets
    leaves = {name: leaf(s[name]) for name in ("x", "a", "b")}
    tp.adapters(**{**s, **leaves}).backward(dout)
    g = torch.Generator(device="cuda").manual_seed(7)
    for name in leaves:
        v = torch.randint(-1, 2, s[name].shape, generator=g, device="cuda").to(torch.bfloat16) * s[name]  # 0, t or 2 t: exact
        up, down = (tp.adapters(**{**s, name: t}).double() for t in (s[name] + v, s[name]))
        diff = ((up - down) * dout.double()).sum()
        grad = leaves[name].grad.double()
        want = (grad * v.double()).sum()
        bound = 2.0 ** -8 * (((up.abs() + down.abs()) * dout.double().abs()).sum() + (grad * v.double()).abs().sum())
        assert abs(diff - want) <= 1.5 * bound, (name, float(diff), float(want), float(bound))


def test_capture_takes_the_calls_but_no_graph(sets):
    import torch

    print("autograd capture", flush=True)
    s, packed, dout = sets
    x = leaf(s["x"])
    out, dx, da, db = torch.empty_like(dout), *(torch.empty_like(s[k]) for k in ("x", "a", "b"))
    want = tp.adapters(**s), *tp.adapters_backward(dout, **s)
    stream = torch.cuda.Stream()

    def both():
        with torch.no_grad():
            tp.adapters(**{**s, "x": x}, out=out)
            tp.adapters_backward(dout, **{**s, "x": x}, dx=dx, da=da, db=db)

    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for call in (lambda: tp.adapters(**{**s, "x": x}), lambda: tp.gated(x, *packed)):
            with pytest.raises(ValueError, match="captured"):
                call()
        both()
    for _ in range(3):
        for t in (out, dx, da, db):
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((out, dx, da, db), want))
