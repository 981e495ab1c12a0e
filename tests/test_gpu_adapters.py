"""GPU parity of adapters() and adapters_backward() against float64.

Bounds are those of tests/rows_reference.py, derived there.
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


def on_gpu(d):
    import torch

    return dict(x=to_dev_bf16(d["x_bits"]), codes=to_dev_codes(d["codes"]), scales=to_dev_bf16(d["scales"]),
                a=to_dev_bf16(d["a_bits"]), b=to_dev_bf16(d["b_bits"]), gain=torch.from_numpy(d["gain"]).cuda(),
                index=torch.from_numpy(d["index"]).cuda()), to_dev_bf16(d["dout_bits"])


def forward(d, bits, out=None):
    s, _ = on_gpu(d)
    got = tp.adapters(bits=bits, out=out, **s)
    return from_dev_bf16(got)


def backward(d, bits):
    s, dout = on_gpu(d)
    dx, da, db = tp.adapters_backward(dout, bits=bits, **s)
    return {"dx": from_dev_bf16(dx), "da": from_dev_bf16(da), "db": from_dev_bf16(db)}


def check_both(d, bits, what):
    value, bound = ref.adapters(d)
    ref.check(what + " out", forward(d, bits), value, bound)
    want = ref.adapters_backward(d)
    got = backward(d, bits)
    for name in ("dx", "da", "db"):
        ref.check(f"{what} {name}", got[name], *want[name])


# n, k: one tile and less, ragged columns, several groups and steps
SHAPES = [(4, 256), (68, 768), (260, 512), (1028, 256), (132, 1792)]


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("m", [1, 17, 130])
def test_shapes(m, n, k, bits):
    print(f"adapters m={m} n={n} k={k} bits={bits}", flush=True)
    rng = np.random.default_rng(1000 * m + n + k + bits)
    d = ref.draw(rng, m, n, k, bits, rank=8, count=3)
    check_both(d, bits, f"m={m} n={n} k={k} bits={bits}")


@pytest.mark.parametrize("rank", [1, 7, 16, 31, 32, 33, 64, 128])
def test_ranks(rank):
    print(f"adapters rank={rank}", flush=True)
    d = ref.draw(np.random.default_rng(rank), 37, 100, 512, 4, rank=rank, count=2)
    check_both(d, 4, f"rank={rank}")


@pytest.mark.parametrize("m", [2, 15, 16, 31, 32, 33, 48, 63, 64, 65, 95, 97, 127, 128, 129, 192, 257, 300])
def test_rows(m):
    print(f"adapters rows m={m}", flush=True)
    d = ref.draw(np.random.default_rng(m), m, 324, 1024, 3, rank=16, count=5)
    check_both(d, 3, f"m={m}")


@pytest.mark.parametrize("kind", ["none", "one", "runs", "outside", "every row its own"])
def test_index_patterns(kind):
    print(f"adapters index {kind}", flush=True)
    m, count = 70, 80
    d = ref.draw(np.random.default_rng(5), m, 132, 512, 2, rank=9, count=count)
    rng = np.random.default_rng(6)
    d["index"] = {
        "none": np.full(m, -1), "one": np.full(m, count - 1), "runs": np.sort(rng.integers(0, 4, m)),
        # values that name no adapter, far ones among them
        "outside": rng.choice([-2**31, -5, -1, 0, 3, count, count + 1, 2**31 - 1], m),
        "every row its own": rng.permutation(count)[:m],
    }[kind].astype(np.int32)
    check_both(d, 2, kind)


def test_rows_without_an_adapter_equal_the_layer_alone():
    # The base rows of a mixed call are the sums of a call without adapters, bit for bit.
    print("adapters base rows", flush=True)
    d = ref.draw(np.random.default_rng(7), 45, 260, 1024, 4, rank=16, count=3)
    mixed = forward(d, 4)
    alone = forward(dict(d, index=np.full(45, -1, np.int32)), 4)
    base = d["index"] < 0
    assert base.any() and np.array_equal(mixed[base], alone[base])


@pytest.fixture
def force_path():
    """Setter for the library's product path; its own choice is restored when the test ends."""
    yield tp.force_path
    tp.force_path(None)


# rows at which a tile, a workgroup's tile or the number of tiles changes
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("m,n,k,rank", [(1, 4, 256, 3), (16, 68, 512, 8), (63, 260, 768, 32), (255, 132, 256, 40),
                                        (256, 516, 512, 16), (257, 1028, 256, 7), (600, 36, 1280, 64)])
def test_weights_decoded_once(force_path, m, n, k, rank, bits):
    print(f"adapters once m={m} n={n} k={k} rank={rank} bits={bits}", flush=True)
    d = ref.draw(np.random.default_rng(m + n + rank), m, n, k, bits, rank=rank, count=3)
    force_path(True)
    check_both(d, bits, f"once m={m} n={n} k={k} rank={rank}")


@pytest.mark.parametrize("m", [300, 641])
def test_weights_decoded_in_the_product_of_many_rows(force_path, m):
    print(f"adapters in the product m={m}", flush=True)
    d = ref.draw(np.random.default_rng(m), m, 388, 1024, 4, rank=16, count=4)
    force_path(False)
    check_both(d, 4, f"in the product m={m}")


def test_weights_decoded_in_several_launches(force_path):
    # 64 and 96 tiles of weights per launch: forward 1540 / 16 = 97 tiles, transposed 2048 / 16 = 128
    print("adapters slabs", flush=True)
    d = ref.draw(np.random.default_rng(31), 70, 1540, 2048, 4, rank=24, count=3)
    force_path(True, 16)
    check_both(d, 4, "slabs")
    force_path(True, 0)
    whole = forward(d, 4)
    force_path(True, 16)
    assert np.array_equal(forward(d, 4), whole)


@pytest.mark.parametrize("path", [False, True])
def test_infinite_weights_of_another_adapter(force_path, path):
    # Rows 0 .. 19 and 20 .. 39 share tiles of 16 rows: the second adapter's
    # infinities must not turn the first's rows into NaN by a zero.
    print(f"adapters infinite path={path}", flush=True)
    d = ref.draw(np.random.default_rng(32), 40, 132, 512, 4, rank=8, count=2)
    d["index"] = np.repeat([0, 1], 20).astype(np.int32)
    force_path(path)
    clean, grads = forward(d, 4), backward(d, 4)
    a_bits, b_bits = d["a_bits"].copy(), d["b_bits"].copy()
    a_bits[1], b_bits[1] = 0x7F80, 0xFF80
    bad = dict(d, a_bits=a_bits, b_bits=b_bits)
    out, bad_grads = forward(bad, 4), backward(bad, 4)
    assert np.array_equal(out[:20], clean[:20])
    assert np.array_equal(bad_grads["dx"][:20], grads["dx"][:20])
    for name in ("da", "db"):
        assert np.array_equal(bad_grads[name][0], grads[name][0])


def test_an_adapters_nan_and_infinity_stay_in_its_rows():
    print("adapters nan", flush=True)
    m, n, k = 40, 68, 512
    d = ref.draw(np.random.default_rng(8), m, n, k, 4, rank=8, count=4)
    clean_out, clean = forward(d, 4), backward(d, 4)
    a_bits, b_bits = d["a_bits"].copy(), d["b_bits"].copy()
    a_bits[1, 3, 5] = 0x7FC0  # NaN
    b_bits[2, 7, 1] = 0x7F80  # +inf
    x_bits = d["x_bits"].copy()
    row = int(np.nonzero(d["index"] == 3)[0][0])
    x_bits[row, 9] = 0x7FC0
    bad = dict(d, a_bits=a_bits, b_bits=b_bits, x_bits=x_bits)
    out, grads = forward(bad, 4), backward(bad, 4)
    fine = ~np.isin(d["index"], [1, 2])
    fine[row] = False
    assert np.array_equal(out[fine], clean_out[fine])
    assert np.array_equal(grads["dx"][fine], clean["dx"][fine])
    assert np.array_equal(grads["da"][0], clean["da"][0])
    assert np.array_equal(grads["db"][0], clean["db"][0])
    assert np.isnan(ref.bf16_bits_to_f32(out[d["index"] == 1])).all()


@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("bits", [2, 3, 4])
def test_extreme_scales(force_path, bits, path):
    # Rows whose scale is zero, subnormal, tiny or huge decode by the page's chain.
    print(f"adapters scales bits={bits} path={path}", flush=True)
    n, k = 132, 512
    force_path(path)
    d = ref.draw(np.random.default_rng(9), 20, n, k, bits, rank=4, count=2)
    for i, s in enumerate([0.0, 2.0 ** -130, 2.0 ** -115, 2.0 ** 112, -0.01]):
        d["scales"][5 + 9 * i] = ref.bf16(np.float32(s))[0][0]
    d["w"] = ref.weights(d["codes"], d["scales"], k, bits)
    value, bound = ref.adapters(d)
    ref.check("scales out", forward(d, bits), value, bound)
    want, got = ref.adapters_backward(d), backward(d, bits)
    ref.check("scales dx", got["dx"], *want["dx"])


def test_gradients_against_differences():
    # <dout, f(x + v) - f(x)> = <dx, v> exactly for this function (linear in x;
    # central differences are exact for A and B too, f being linear in each).
    print("adapters differences", flush=True)
    rng = np.random.default_rng(10)
    d = ref.draw(rng, 33, 68, 512, 3, rank=5, count=2)
    got = {k: ref.bf16_bits_to_f32(v).astype(np.float64) for k, v in backward(d, 3).items()}
    want = ref.adapters_backward(d)

    def f(x, a, b):
        out = x @ d["w"].T
        for i in range(2):
            of = d["index"] == i
            out[of] += d["gain"][i] * (x[of] @ a[i].T @ b[i].T)
        return out

    x, a, b = d["x"], d["a"], d["b"]
    for name, step in (("dx", lambda v: (v, 0, 0)), ("da", lambda v: (0, v, 0)), ("db", lambda v: (0, 0, v))):
        v = rng.standard_normal(got[name].shape)
        vx, va, vb = step(v)
        diff = ((f(x + vx, a + va, b + vb) - f(x - vx, a - va, b - vb)) / 2 * d["dout"]).sum()
        assert abs(diff - (got[name] * v).sum()) <= (want[name][1] * np.abs(v)).sum()


def test_rows_behind_the_last_are_left_alone():
    import torch

    print("adapters rows behind", flush=True)
    m, n, k, bits = 21, 36, 256, 4
    d = ref.draw(np.random.default_rng(11), m, n, k, bits, rank=3, count=2)
    s, dout = on_gpu(d)
    big = torch.full((m + 8, n), 7.0, dtype=torch.bfloat16, device="cuda")
    tp.adapters(bits=bits, out=big[:m], **s)
    dx = torch.full((m + 8, k), 7.0, dtype=torch.bfloat16, device="cuda")
    da = torch.full((4, 3, k), 7.0, dtype=torch.bfloat16, device="cuda")
    db = torch.full((4, n, 3), 7.0, dtype=torch.bfloat16, device="cuda")
    tp.adapters_backward(dout, bits=bits, dx=dx[:m], da=da[:2], db=db[:2], **s)
    torch.cuda.synchronize()
    for t, used in ((big, m), (dx, m), (da, 2), (db, 2)):
        assert bool((t[used:] == 7.0).all()) and not bool((t[:used] == 7.0).all())


def test_the_same_call_twice_gives_the_same_bits():
    print("adapters repeat", flush=True)
    d = ref.draw(np.random.default_rng(12), 150, 516, 1536, 4, rank=24, count=6)
    one, two = backward(d, 4), backward(d, 4)
    assert all(np.array_equal(one[k], two[k]) for k in one)
    assert np.array_equal(forward(d, 4), forward(d, 4))


def test_another_stream_and_a_captured_graph():
    import torch

    print("adapters graph", flush=True)
    bits = 4
    d = ref.draw(np.random.default_rng(13), 50, 260, 1024, bits, rank=16, count=3)
    e = ref.draw(np.random.default_rng(14), 50, 260, 1024, bits, rank=16, count=3)
    s, dout = on_gpu(d)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = torch.empty((50, 260), dtype=torch.bfloat16, device="cuda")
    dx, da, db = (torch.empty_like(t) for t in (s["x"], s["a"], s["b"]))

    def both():
        tp.adapters(bits=bits, out=out, **s)
        tp.adapters_backward(dout, bits=bits, dx=dx, da=da, db=db, **s)

    with torch.cuda.stream(stream):
        both()  # the first call of a shape allocates
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        both()
    for data in (e, d, e):
        s2, dout2 = on_gpu(data)
        for key in s:
            s[key].copy_(s2[key])
        dout.copy_(dout2)
        torch.cuda.synchronize()
        for t in (out, dx, da, db):
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        want = backward(data, bits)
        assert np.array_equal(from_dev_bf16(out), forward(data, bits))
        for name, t in (("dx", dx), ("da", da), ("db", db)):
            assert np.array_equal(from_dev_bf16(t), want[name]), name


def test_two_streams_at_once():
    import torch

    print("adapters two streams", flush=True)
    bits = 4
    sets = [on_gpu(ref.draw(np.random.default_rng(20 + i), 40 + 30 * i, 1028, 1024, bits, rank=16, count=3)) for i in range(2)]
    alone = []
    for s, dout in sets:
        alone.append([t.clone() for t in (tp.adapters(bits=bits, **s), *tp.adapters_backward(dout, bits=bits, **s))])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(5):
        for i, (s, dout) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i] = (tp.adapters(bits=bits, **s), *tp.adapters_backward(dout, bits=bits, **s))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(got[i], alone[i]))


@pytest.mark.parametrize("path", [False, True])
def test_infinities_stay_infinities(force_path, path):
    # An infinite t, u, x, dout or factor gives the infinity (or the NaN) that
    # the formula gives: a float32 number enters these products in two halves.
    print(f"adapters infinities path={path}", flush=True)
    d = ref.draw(np.random.default_rng(41), 40, 68, 512, 4, rank=8, count=4)
    d["index"] = np.arange(40, dtype=np.int32) % 5
    for name, at, value in (("a", (1, 3, 5), np.inf), ("b", (2, 7, 1), -np.inf), ("x", (3, 9), np.inf),
                            ("dout", (5, 11), -np.inf)):
        d[name][at] = value
        d[name + "_bits"][at] = 0x7F80 if value > 0 else 0xFF80
    force_path(path)
    with np.errstate(invalid="ignore"):
        check_both(d, 4, f"infinities path={path}")
        value = {"out": ref.adapters(d)[0], **{k: v[0] for k, v in ref.adapters_backward(d).items()}}
    got = {"out": forward(d, 4), **backward(d, 4)}
    for name, v in value.items():
        at = np.isinf(v)
        assert at.any() and np.array_equal(ref.bf16_bits_to_f32(got[name])[at], v[at]), name


@pytest.mark.parametrize("mode", ["global", "relaxed"])
def test_a_capture_without_a_call_before_it_is_refused(mode):
    import torch

    print(f"adapters first call in a capture, {mode}", flush=True)
    d = ref.draw(np.random.default_rng(42), 50, 260, 1024, 4, rank=16, count=3)
    s, _ = on_gpu(d)
    want = forward(d, 4)
    out = torch.zeros((50, 260), dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    # Streams come from a pool, so one that an earlier test used has a
    # workspace: many rows need more than any of them.
    rows = 1 << 16
    big = dict(s, x=s["x"].repeat(rows // 50, 1), index=s["index"].repeat(rows // 50))
    big_out = torch.zeros((rows // 50 * 50, 260), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(tp.TrellisError):
        with torch.cuda.graph(graph, stream=stream, capture_error_mode=mode):
            out.add_(0)
            tp.adapters(bits=4, out=big_out, **big)
    torch.cuda.synchronize()
    for _ in range(2):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            tp.adapters(bits=4, out=out, **s)
        torch.cuda.synchronize()
        assert np.array_equal(from_dev_bf16(out), want)
    with torch.cuda.stream(stream):
        tp.adapters(bits=4, out=big_out, **big)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream, capture_error_mode=mode):
        tp.adapters(bits=4, out=out, **s)
    for _ in range(2):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(from_dev_bf16(out), want)
