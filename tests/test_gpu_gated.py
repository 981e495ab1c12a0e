"""GPU parity of gated() and gated_backward() against float64, and of a run of
them with the adapters as a training step calls them.

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


def draw(seed, m, n, k, bits):
    rng = np.random.default_rng(seed)
    g, u = ref.draw(rng, m, n, k, bits), ref.draw(rng, m, n, k, bits)
    std = 0.0127 * k ** 0.5
    d = {"x_bits": g["x_bits"], "x": g["x"], "gate_w": g, "up_w": u, "k": k, "bits": bits}
    for name, scale in (("gate", std), ("up", std), ("dh", 1.0)):
        d[name + "_bits"], d[name] = ref.bf16(rng.standard_normal((m, n)) * scale)
    return d


def packed(d):
    return (to_dev_codes(d["gate_w"]["codes"]), to_dev_bf16(d["gate_w"]["scales"]), to_dev_codes(d["up_w"]["codes"]),
            to_dev_bf16(d["up_w"]["scales"]), d["bits"])


def check_forward(d, what):
    h, gate, up = tp.gated(to_dev_bf16(d["x_bits"]), *packed(d), keep=True)
    plain = tp.gated(to_dev_bf16(d["x_bits"]), *packed(d))
    want = ref.gated(d["x"], d["gate_w"]["w"], d["up_w"]["w"])
    for name, t in (("h", h), ("gate", gate), ("up", up)):
        ref.check(f"{what} {name}", from_dev_bf16(t), *want[name])
    assert np.array_equal(from_dev_bf16(plain), from_dev_bf16(h))


def check_backward(d, what):
    dx, dgate, dup = tp.gated_backward(to_dev_bf16(d["dh_bits"]), to_dev_bf16(d["gate_bits"]),
                                       to_dev_bf16(d["up_bits"]), *packed(d))
    want = ref.gated_grads(d["dh"], d["gate"], d["up"])
    got = {}
    for name, t in (("dgate", dgate), ("dup", dup)):
        ref.check(f"{what} {name}", from_dev_bf16(t), *want[name])
        got[name] = ref.bf16_bits_to_f32(from_dev_bf16(t)).astype(np.float64)
    # dx is the product of the rounded gradients, as documented
    both = np.concatenate([got["dgate"], got["dup"]], 1)
    w = np.concatenate([d["gate_w"]["w"], d["up_w"]["w"]], 0)
    value, err = ref.product(both, w.T)
    ref.check(f"{what} dx", from_dev_bf16(dx), value, ref.rounded(err, value))


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("n,k", [(4, 256), (68, 768), (260, 512), (1028, 256), (132, 1792)])
@pytest.mark.parametrize("m", [1, 17, 130])
def test_shapes(m, n, k, bits):
    print(f"gated m={m} n={n} k={k} bits={bits}", flush=True)
    d = draw(2000 * m + n + k + bits, m, n, k, bits)
    check_forward(d, f"m={m} n={n} k={k} bits={bits}")
    check_backward(d, f"m={m} n={n} k={k} bits={bits}")


@pytest.mark.parametrize("m", [2, 15, 16, 32, 33, 64, 65, 95, 97, 128, 129, 257, 300])
def test_rows(m):
    print(f"gated rows m={m}", flush=True)
    d = draw(m, m, 324, 1024, 4)
    check_forward(d, f"m={m}")
    check_backward(d, f"m={m}")


@pytest.fixture
def force_path():
    """Setter for the library's product path; its own choice is restored when the test ends."""
    yield tp.force_path
    tp.force_path(None)


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("m,n,k", [(1, 4, 256), (16, 68, 512), (255, 132, 256), (257, 1028, 256), (600, 36, 1280)])
def test_weights_decoded_once(force_path, m, n, k, bits):
    print(f"gated once m={m} n={n} k={k} bits={bits}", flush=True)
    d = draw(m + n + k, m, n, k, bits)
    force_path(True)
    check_forward(d, f"once m={m} n={n} k={k}")
    check_backward(d, f"once m={m} n={n} k={k}")


@pytest.mark.parametrize("m", [300, 641])
def test_weights_decoded_in_the_product_of_many_rows(force_path, m):
    print(f"gated in the product m={m}", flush=True)
    d = draw(m, m, 388, 1024, 4)
    force_path(False)
    check_forward(d, f"in the product m={m}")
    check_backward(d, f"in the product m={m}")


def test_weights_decoded_in_several_launches(force_path):
    print("gated slabs", flush=True)
    d = draw(9, 70, 1540, 2048, 4)
    force_path(True, 16)
    check_forward(d, "slabs")
    check_backward(d, "slabs")


def test_far_gates_keep_their_limits():
    # Gates at which exp overflows: silu and its derivative reach their limits.
    print("gated far gates", flush=True)
    d = draw(3, 4, 36, 256, 4)
    far = np.array([200.0, -200.0, 80.0, -80.0, 0.0, -0.0, 30.0, -30.0], np.float32)
    gate = np.tile(far, 18)[: 4 * 36].reshape(4, 36)
    d["gate_bits"], d["gate"] = ref.bf16(gate)
    check_backward(d, "far gates")


def test_differences():
    # The gradient of sum(dh * h) along a direction, by central differences in
    # 64 bits (step 1e-4: the error of the differences is about 1e-8 relative).
    print("gated differences", flush=True)
    d = draw(4, 21, 68, 512, 3)
    want = ref.gated(d["x"], d["gate_w"]["w"], d["up_w"]["w"])
    for name in ("gate", "up"):
        d[name + "_bits"], d[name] = ref.bf16(want[name][0])
    dx = tp.gated_backward(to_dev_bf16(d["dh_bits"]), to_dev_bf16(d["gate_bits"]), to_dev_bf16(d["up_bits"]), *packed(d))[0]
    got = ref.bf16_bits_to_f32(from_dev_bf16(dx)).astype(np.float64)
    v = np.random.default_rng(5).standard_normal(d["x"].shape)

    def f(x):
        g, u = x @ d["gate_w"]["w"].T, x @ d["up_w"]["w"].T
        return (g * ref.sigmoid(g) * u * d["dh"]).sum()

    diff = (f(d["x"] + 1e-4 * v) - f(d["x"] - 1e-4 * v)) / 2e-4
    # The kept projections are rounded (2^-8 of each): with |silu''| <= 0.5 the
    # gradients move by at most |dh| (|up| 0.5 |gate| + 1.1 |up|) 2^-8 and
    # |dh| 1.1 |gate| 2^-8; each is then rounded (2^-8), and so is dx.
    g, u, dh = np.abs(want["gate"][0]), np.abs(want["up"][0]), np.abs(d["dh"])
    e = 2.0 ** -8
    eg = dh * (u * 0.5 * g + 1.1 * u) * e + e * 1.1 * dh * u
    eu = dh * 1.1 * g * e + e * dh * g
    bound = eg @ np.abs(d["gate_w"]["w"]) + eu @ np.abs(d["up_w"]["w"]) + e * np.abs(got) + 1e-5
    assert abs(diff - (got * v).sum()) <= 1.01 * (bound * np.abs(v)).sum()


def test_repeat_graph_and_stream():
    import torch

    print("gated graph", flush=True)
    d, e = draw(5, 70, 260, 1024, 4), draw(6, 70, 260, 1024, 4)

    def tensors(q):
        return [to_dev_bf16(q[n]) for n in ("x_bits", "gate_bits", "up_bits", "dh_bits")]

    weights = packed(d)
    x, gate, up, dh = tensors(d)
    out = torch.empty_like(gate)
    dx, dgate, dup = torch.empty_like(x), torch.empty_like(gate), torch.empty_like(gate)

    def both():
        tp.gated(x, *weights, out=out)
        tp.gated_backward(dh, gate, up, *weights, dx=dx, dgate=dgate, dup=dup)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        both()
    for q in (e, d, e):
        for t, new in zip((x, gate, up, dh), tensors(q)):
            t.copy_(new)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        eager = (tp.gated(x, *weights), *tp.gated_backward(dh, gate, up, *weights))
        assert all(torch.equal(p, r) for p, r in zip((out, dx, dgate, dup), eager))


def test_a_training_step_of_the_mlp():
    """The block as it is used: the gated projections, the down projection with
    its adapters, and back; every step against float64 on what it was given."""
    print("mlp step", flush=True)
    m, k, n, bits, rank, count = 75, 512, 1024, 4, 12, 3
    d = draw(7, m, n, k, bits)
    rng = np.random.default_rng(8)
    down = ref.draw(rng, m, k, n, bits, rank=rank, count=count)  # [k, n]: back to the block's width
    import torch

    h, gate, up = tp.gated(to_dev_bf16(d["x_bits"]), *packed(d), keep=True)
    s = dict(codes=to_dev_codes(down["codes"]), scales=to_dev_bf16(down["scales"]), bits=bits,
             a=to_dev_bf16(down["a_bits"]), b=to_dev_bf16(down["b_bits"]), gain=torch.from_numpy(down["gain"]).cuda(),
             index=torch.from_numpy(down["index"]).cuda())
    y = tp.adapters(h, **s)
    dy = to_dev_bf16(down["dout_bits"])
    dh, da, db = tp.adapters_backward(dy, h, **s)
    dx, dgate, dup = tp.gated_backward(dh, gate, up, *packed(d))
    torch.cuda.synchronize()

    want = ref.gated(d["x"], d["gate_w"]["w"], d["up_w"]["w"])
    for name, t in (("h", h), ("gate", gate), ("up", up)):
        ref.check(f"step {name}", from_dev_bf16(t), *want[name])
    down["x"] = ref.bf16_bits_to_f32(from_dev_bf16(h)).astype(np.float64)
    ref.check("step y", from_dev_bf16(y), *ref.adapters(down))
    grads = ref.adapters_backward(down)
    for name, t in (("dx", dh), ("da", da), ("db", db)):
        ref.check(f"step {name}", from_dev_bf16(t), *grads[name])
    f64 = {name: ref.bf16_bits_to_f32(from_dev_bf16(t)).astype(np.float64)
           for name, t in (("dh", dh), ("gate", gate), ("up", up), ("dgate", dgate), ("dup", dup))}
    for name, t in ref.gated_grads(f64["dh"], f64["gate"], f64["up"]).items():
        ref.check(f"step {name}", from_dev_bf16({"dgate": dgate, "dup": dup}[name]), *t)
    value, err = ref.product(np.concatenate([f64["dgate"], f64["dup"]], 1),
                             np.concatenate([d["gate_w"]["w"], d["up_w"]["w"]], 0).T)
    ref.check("step dx", from_dev_bf16(dx), value, ref.rounded(err, value))
