"""The losses and the embedding as a training program uses them: recorded by
autograd, one after the other with the fine-tuned layers, on several streams, in
captured graphs, and at sizes whose offsets pass 32 bits."""
import numpy as np
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests import rows_reference as rows
from tests import vocabulary_reference as ref
from tests.helpers import from_dev_bf16, to_dev_bf16, to_dev_codes
from workloads import bf16_bits_to_f32

pytestmark = pytest.mark.gpu

M, N, K, BITS, EXTRA, TOP = 45, 516, 512, 4, 6, 3


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tp.load_library()


def dev(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.fixture
def parts():
    """One packed vocabulary matrix, embedding and output layer at once, with everything the calls take."""
    rng = np.random.default_rng(5)
    d = ref.draw(rng, M, N, K, BITS, top=TOP)
    index = d["index"].copy()
    index[::7], index[1::7, 1:] = -1, N + 3  # padding rows, short lists
    tokens = rng.integers(0, N + EXTRA, M).astype(np.int32)
    tokens[:6] = N + np.arange(6)
    tokens[-5:] = -1  # a padded batch
    return dict(d=d, packed=(to_dev_codes(d["codes"]), to_dev_bf16(d["scales"]), BITS), x=to_dev_bf16(d["x_bits"]),
                target=dev(index[:, 0]), index=dev(index), logits=dev(d["logits"]), tokens=dev(tokens),
                extra=to_dev_bf16(ref.bf16(rng.standard_normal((EXTRA, K)))[0]), host_index=index, host_tokens=tokens)


def leaf(t):
    return t.clone().requires_grad_()


def embed(p, extra):
    codes, scales, bits = p["packed"]
    return tp.embed(p["tokens"], codes, scales, K, bits, scale=3.0, extra=extra)


@pytest.mark.parametrize("what", ["cross_entropy", "distill"])
def test_losses_under_autograd(parts, what):
    import torch

    print(f"autograd {what}", flush=True)
    p = parts
    lists = (p["target"],) if what == "cross_entropy" else (p["index"], p["logits"], 1.7)
    call = getattr(tp, what)
    want = call(p["x"], *p["packed"], *lists, keep=True)
    dloss = torch.randn(M, device="cuda")
    x = leaf(p["x"])
    loss, lse = call(x, *p["packed"], *lists)
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1]) and loss.requires_grad
    loss.backward(dloss)
    assert torch.equal(x.grad, tp.loss_backward(dloss, want[2]))
    # a mean: an expanded gradient; the kept dx beside it
    x = leaf(p["x"])
    loss, lse, dx = call(x, *p["packed"], *lists, keep=True)
    assert torch.equal(dx, want[2]) and not dx.requires_grad
    loss.mean().backward()
    assert torch.equal(x.grad, tp.loss_backward(torch.full((M,), 1 / M, device="cuda"), want[2]))
    # lse carries no gradient, alone or beside the loss; without gradients nothing is recorded
    loss, lse = call(leaf(p["x"]), *p["packed"], *lists)
    with pytest.raises(RuntimeError, match="lse"):
        (loss.sum() + lse.sum()).backward()
    with torch.no_grad():
        assert not call(leaf(p["x"]), *p["packed"], *lists)[0].requires_grad
    scales = p["packed"][1].clone().requires_grad_()
    with pytest.raises(ValueError, match="scales"):
        call(p["x"], p["packed"][0], scales, BITS, *lists)
    if what == "distill":
        with pytest.raises(ValueError, match="logits"):
            call(p["x"], *p["packed"], p["index"], leaf(p["logits"]))


def test_embedding_under_autograd(parts):
    import torch

    print("autograd embed", flush=True)
    p = parts
    extra = leaf(p["extra"])
    out = embed(p, extra)
    assert torch.equal(out, embed(p, p["extra"]))
    dout = torch.randn(M, K, device="cuda").bfloat16()
    out.backward(dout)
    assert torch.equal(extra.grad, tp.embed_backward(dout, p["tokens"], N, EXTRA, scale=3.0))
    extra = leaf(p["extra"])
    embed(p, extra).sum().backward()
    assert torch.equal(extra.grad, tp.embed_backward(torch.ones_like(dout), p["tokens"], N, EXTRA, scale=3.0))
    with pytest.raises(ValueError, match="out="):
        tp.embed(p["tokens"], *p["packed"][:2], K, BITS, extra=leaf(p["extra"]), out=torch.empty_like(dout))


def step(p, layer, extra, a, b, lists, temperature):
    """Embedding, a gated block brought back to the model's width, a projection with adapters, a distillation loss."""
    import torch

    h = tp.gated(embed(p, extra), *layer["gated"])
    h = torch.nn.functional.pad(h, (0, K - h.shape[1]))
    y = tp.adapters(h, layer["codes"], layer["scales"], BITS, a, b, layer["gain"], layer["index"])
    return tp.distill(y, *p["packed"], *lists, temperature=temperature)[0]


def test_a_whole_step_on_two_streams(parts):
    """The calls in a row, against the same calls made by hand; then on two streams at once, three times over."""
    import torch

    print("whole step", flush=True)
    p, rng = parts, np.random.default_rng(8)
    d, e = rows.draw(rng, M, 260, K, BITS), rows.draw(rng, M, 260, K, BITS)
    w = rows.draw(rng, M, K, K, BITS, rank=8, count=2)
    layer = dict(gated=(to_dev_codes(d["codes"]), to_dev_bf16(d["scales"]), to_dev_codes(e["codes"]),
                        to_dev_bf16(e["scales"]), BITS), codes=to_dev_codes(w["codes"]), scales=to_dev_bf16(w["scales"]),
                 gain=dev(w["gain"]), index=dev(w["index"]))
    a0, b0 = to_dev_bf16(w["a_bits"]), to_dev_bf16(w["b_bits"])
    lists = p["index"], p["logits"]
    dloss = torch.rand(M, device="cuda")
    with torch.no_grad():
        x = embed(p, p["extra"])
        h, gate, up = tp.gated(x, *layer["gated"], keep=True)
        wide = torch.nn.functional.pad(h, (0, K - h.shape[1]))
        args = layer["codes"], layer["scales"], BITS, a0, b0, layer["gain"], layer["index"]
        y = tp.adapters(wide, *args)
        loss, _, dy = tp.distill(y, *p["packed"], *lists, temperature=1.5, keep=True)
        dh, da, db = tp.adapters_backward(tp.loss_backward(dloss, dy), wide, *args)
        dx = tp.gated_backward(dh[:, :260].contiguous(), gate, up, *layer["gated"])[0]
        dextra = tp.embed_backward(dx, p["tokens"], N, EXTRA, scale=3.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                leaves = leaf(p["extra"]), leaf(a0), leaf(b0)
                out = step(p, layer, *leaves, lists, 1.5)
                got.append((out, *torch.autograd.grad(out, leaves, dloss)))
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(u, v) for u, v in zip(g, (loss, dextra, da, db)))


@pytest.mark.parametrize("path", [(None, 0), (False, 0), (True, 0), (True, 16)])
def test_captured_calls(parts, path):
    """All calls in one graph, replayed on new inputs between eager calls on the same stream."""
    import torch

    print(f"captured {path}", flush=True)
    p = parts
    tp.force_path(*path)
    try:
        x, tokens, dloss = p["x"].clone(), p["tokens"].clone(), torch.rand(M, device="cuda")
        codes, scales, bits = p["packed"]

        def calls():
            with torch.no_grad():
                ce = tp.cross_entropy(x, *p["packed"], p["target"], keep=True)
                ds = tp.distill(x, *p["packed"], p["index"], p["logits"], temperature=2.0, keep=True)
                dx = tp.loss_backward(dloss, ce[2])
                e = tp.embed(tokens, codes, scales, K, bits, extra=p["extra"])
                return (*ce, *ds, dx, e, tp.embed_backward(e, tokens, N, EXTRA))

        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            calls()  # the stream's workspace
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = calls()
            with pytest.raises(ValueError, match="captured"):
                tp.cross_entropy(leaf(p["x"]), *p["packed"], p["target"])
        for rep in range(4):
            x.copy_(p["x"].roll(rep, 0))
            tokens.copy_(p["tokens"].roll(rep, 0))
            for o in outs:
                o.fill_(float("nan"))
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            with torch.cuda.stream(stream):
                want = calls()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(got, want)), rep
    finally:
        tp.force_path(None)


def test_a_capture_that_would_allocate_is_refused(parts):
    import torch

    print("capture without workspace", flush=True)
    p, stream = parts, torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        keep = p["x"] + 0
        with pytest.raises(tp.TrellisError):
            tp.cross_entropy(p["x"], *p["packed"], p["target"])
        with pytest.raises(tp.TrellisError):
            tp.embed_backward(p["x"], p["tokens"], N, EXTRA)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(keep, p["x"])


def plain_loss(x, w, target, dtype):
    import torch

    l = x.to(dtype) @ w.to(dtype).T
    lse = torch.logsumexp(l, 1)
    keep = (target >= 0) & (target < w.shape[0])
    at = target.clamp(0, w.shape[0] - 1).long()[:, None]
    loss = torch.where(keep, lse - l.gather(1, at)[:, 0], 0.0)
    d = (l - lse[:, None]).exp_()
    d.scatter_add_(1, at, torch.full_like(lse[:, None], -1.0))
    return loss, lse, (d * keep[:, None]) @ w.to(dtype)


@pytest.mark.parametrize("m,n,path", [(5000, 131072, (True, 0)), (2100, 131076, (False, 0)), (700, 1 << 20, (None, 0))])
def test_chunks_of_rows(m, n, path):
    """More rows than a chunk's workspace takes, of large vocabularies: every row against the same rows' formula in
    float64 on the GPU. Bounds as in tests/vocabulary_reference.py, with N E24 for the sums over the vocabulary."""
    import torch

    print(f"chunks {m} {n} {path}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    k, bits = 256, 2
    codes = torch.randint(-2**31, 2**31, (n, k * bits // 32), generator=g, device="cuda", dtype=torch.int32)
    scales = (torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005).bfloat16()
    x = (torch.randn(m, k, generator=g, device="cuda") * 4).bfloat16()
    target = torch.randint(-1, n + 1, (m,), generator=g, device="cuda", dtype=torch.int32)
    w = tp.decode(codes, scales, k, bits)
    try:
        tp.force_path(*path)
        got = tp.cross_entropy(x, codes, scales, bits, target, keep=True)
        short = tp.cross_entropy(x, codes, scales, bits, target)
    finally:
        tp.force_path(None)
    e24 = 2.0 ** -24
    largest = w.double().abs().max()
    for r0 in list(range(0, m, 512)):
        r = slice(r0, min(m, r0 + 512))
        loss, lse, dx = plain_loss(x[r], w, target[r], torch.float64)
        el = k * e24 * (x[r].double().abs().sum(1) * largest) + 4 * e24 * 40
        bound = 2 * el + 2.0 ** -17 + 8 * e24 * lse.abs()
        for o in (got, short):
            assert ((o[0][r] - loss).abs() <= 2 * bound).all() and ((o[1][r] - lse).abs() <= bound).all()
        # dx: sum_v p_v |W_v| + |W_target| <= 2 max|W|, each term off by 2^-8 (twice, where p is kept apart) and the logits' errors
        off = (got[2][r].double() - dx).abs()
        assert (off <= 2 * largest * (2 * 2.0 ** -8 + 2 * bound[:, None]) + 2.0 ** -8 * dx.abs()).all()
        # and close by the row's norm: the roundings' signs differ
        assert (off.norm(dim=1) <= 2.0 ** -7 * dx.norm(dim=1) + 1e-6).all()


def test_offsets_past_32_bits():
    """2^20 rows of 2304 columns: more than 2^31 elements of the embedding and of its gradient's input."""
    import torch

    print("offsets past 32 bits", flush=True)
    m, k, n, count = 1 << 20, 2304, 1000, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(-2**31, 2**31, (n, k * 2 // 32), generator=g, device="cuda", dtype=torch.int32)
    scales = (torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005).bfloat16()
    extra = torch.randn(count, k, generator=g, device="cuda").bfloat16()
    tokens = torch.randint(-1, n + count, (m,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.cat([tp.decode(codes, scales, k, 2), extra, torch.zeros_like(extra[:1])])
    out = tp.embed(tokens, codes, scales, k, 2, extra=extra)
    for r in (slice(0, 1000), slice(m - 1000, m), slice(931000, 933000)):  # 2^31 / 2304 = 932067
        assert torch.equal(out[r], table[tokens[r].long()])
    # small whole numbers: every float32 sum is exact, whatever its order
    dout = torch.randint(-2, 3, (m, k), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    got = tp.embed_backward(dout, tokens, n, count)
    want = torch.zeros(count, k, device="cuda", dtype=torch.float64)
    for r0 in range(0, m, 1 << 17):
        t = tokens[r0:r0 + (1 << 17)].long() - n
        at = (t >= 0).nonzero()[:, 0]
        want.index_add_(0, t[at], dout[r0:r0 + (1 << 17)][at].double())
    assert torch.equal(got, want.bfloat16())


def test_loss_offsets_past_32_bits():
    """2^20 rows of 2304 columns in several chunks: more than 2^31 elements of x and of its gradient."""
    import torch

    print("loss offsets past 32 bits", flush=True)
    m, k, n = 1 << 20, 2304, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    codes = torch.randint(-2**31, 2**31, (n, k * 4 // 32), generator=g, device="cuda", dtype=torch.int32)
    scales = (torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005).bfloat16()
    x = torch.randn(m, k, generator=g, device="cuda", dtype=torch.bfloat16)
    target = torch.randint(-1, n, (m,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse, dx = tp.cross_entropy(x, codes, scales, 4, target, keep=True)
    w = tp.decode(codes, scales, k, 4)
    largest = w.double().abs().max()
    for r in (slice(0, 500), slice(932000, 932500), slice(m - 500, m)):
        want = plain_loss(x[r], w, target[r], torch.float64)
        el = k * 2.0 ** -24 * x[r].double().abs().sum(1) * largest
        bound = 2 * el + 2.0 ** -17
        assert ((loss[r] - want[0]).abs() <= 2 * bound).all() and ((lse[r] - want[1]).abs() <= bound).all()
        off = (dx[r].double() - want[2]).abs()
        assert (off <= 2 * largest * (2 * 2.0 ** -8 + 2 * bound[:, None]) + 2.0 ** -8 * want[2].abs()).all()
