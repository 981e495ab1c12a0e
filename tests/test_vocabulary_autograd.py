"""What autograd records for the losses and for embed(), and what it learns of
outputs that the caller gives, on the CPU: the raw calls are replaced by the
plain formulas on host tensors."""
import ctypes

import pytest
import torch

import trellis_coded_bit_prefill_amd as tp

M, N, K, BITS, COUNT = 6, 8, 256, 2, 3


def draw(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def put(address, value, dtype=torch.bfloat16):
    value = value.to(dtype).contiguous()
    ctypes.memmove(address, value.data_ptr(), value.numel() * value.element_size())


def at(address, *shape, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype)
    ctypes.memmove(out.data_ptr(), address, out.numel() * out.element_size())
    return out


@pytest.fixture
def plain(monkeypatch):
    """The calls' inputs; a layer's gradient stands in for each kernel's."""
    w = draw(N, K, seed=1)
    t = {"x": draw(M, K, seed=2), "codes": torch.zeros((N, K * BITS // 32), dtype=torch.int32), "scales": draw(N),
         "target": torch.tensor([1, -1, 0, 7, 1, 5], dtype=torch.int32),
         "index": torch.tensor([[1, 2], [-1, -1], [0, 3], [7, 7], [1, -1], [5, 6]], dtype=torch.int32),
         "logits": torch.randn(M, 2), "tokens": torch.tensor([0, 7, 8, 10, 8, -1], dtype=torch.int32),
         "extra": draw(COUNT, K, seed=3)}

    def losses(x, m, loss, lse, dx, scale):
        l = at(x, m, K).double() @ w.double().T
        put(loss, scale * l.square().sum(1), torch.float32)
        put(lse, l.logsumexp(1), torch.float32)
        if dx:
            put(dx, 2 * scale * l @ w.double())

    def cross_entropy_raw(x, m, codes, scales, g, target, loss, lse, dx, stream):
        losses(x, m, loss, lse, dx, 1)

    def distill_raw(x, m, codes, scales, g, index, logits, top, temperature, loss, lse, dx, stream):
        losses(x, m, loss, lse, dx, temperature)

    def loss_backward_raw(dloss, dx, m, k, out, stream):
        put(out, at(dloss, m, dtype=torch.float32)[:, None] * at(dx, m, k).float())

    def embed_raw(tokens, m, codes, scales, g, scale, extra, count, out, stream):
        rows = [at(extra, count, g.k)] if count else []
        table = torch.cat([w, *rows, torch.zeros(1, g.k, dtype=torch.bfloat16)])
        token = at(tokens, m, dtype=torch.int32).long()
        put(out, table[torch.where((token < 0) | (token >= N + count), N + count, token)].float() * scale)

    def embed_backward_raw(dout, tokens, m, k, first, count, scale, dextra, stream):
        token = at(tokens, m, dtype=torch.int32).long() - first
        put(dextra, scale * ((token == torch.arange(count)[:, None]).double() @ at(dout, m, k).double()))

    for f in (cross_entropy_raw, distill_raw, loss_backward_raw, embed_raw, embed_backward_raw):
        monkeypatch.setattr(tp, f.__name__, f)
    monkeypatch.setattr(tp, "_stream_handle", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    check = tp._check_tensor
    monkeypatch.setattr(tp, "_check_tensor", lambda name, v, *r: check(name, v, *r) if not isinstance(v, torch.Tensor) else None)
    return t


def leaf(v):
    return v.clone().requires_grad_()


LOSSES = {"cross_entropy": lambda t, x, **kw: tp.cross_entropy(x, t["codes"], t["scales"], BITS, t["target"], **kw),
          "distill": lambda t, x, **kw: tp.distill(x, t["codes"], t["scales"], BITS, t["index"], t["logits"], 2.0, **kw)}


@pytest.mark.parametrize("what", list(LOSSES))
def test_gradients(plain, what):
    dx = LOSSES[what](plain, plain["x"], keep=True)[2]
    x, dloss = leaf(plain["x"]), torch.randn(M)
    LOSSES[what](plain, x)[0].backward(dloss)
    assert torch.equal(x.grad, tp.loss_backward(dloss, dx))
    x = leaf(plain["x"])
    loss, _, kept = LOSSES[what](plain, x, keep=True)
    assert torch.equal(kept, dx)
    other = tp.loss_backward(dloss, kept)  # a buffer of its own: the kept one stays as it is
    loss.backward(dloss)
    assert torch.equal(x.grad, other)


@pytest.mark.parametrize("what", list(LOSSES))
def test_a_kept_gradient_that_is_overwritten(plain, what):
    """A recorded call's dx is what its backward pass multiplies: written over, the pass raises."""
    loss, _, dx = LOSSES[what](plain, leaf(plain["x"]), keep=True)
    assert tp.loss_backward(torch.full((M,), 3.0), dx, out=dx) is dx
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    # not recorded: nothing else holds it
    _, _, dx = LOSSES[what](plain, plain["x"], keep=True)
    want = tp.loss_backward(torch.full((M,), 3.0), dx)
    assert torch.equal(tp.loss_backward(torch.full((M,), 3.0), dx, out=dx), want)


def test_given_outputs_are_known_to_be_written(plain, monkeypatch):
    """Every call with an output of the caller's moves its version counter, once the call is made."""
    t = plain
    for name in ("decode_raw", "prefill_raw", "prefill_noalloc_raw", "matvec_raw", "prefill_packed_raw", "gate_up_raw",
                 "adapters_raw", "adapters_backward_raw", "gated_raw", "gated_backward_raw"):
        monkeypatch.setattr(tp, name, lambda *a: None)
    layer, two = (t["codes"], t["scales"], BITS), (t["codes"], t["scales"]) * 2 + (BITS,)
    wide, narrow, small = (lambda: draw(M, K)), (lambda: draw(M, N)), (lambda: draw(COUNT, K))
    a, b = draw(2, 4, K), draw(2, N, 4)
    set_ = a, b, torch.ones(2), torch.zeros(M, dtype=torch.int32)
    gate = draw(M, N)
    calls = [
        (lambda o: tp.decode(*layer[:2], K, BITS, out=o), [draw(N, K)]),
        (lambda o: tp.prefill(t["x"], *layer, out=o), [narrow()]),
        (lambda o: tp.prefill_noalloc(t["x"], *layer, out=o), [narrow()]),
        (lambda o: tp.matvec(t["x"], *layer, out=o), [narrow()]),
        (lambda *o: tp.prefill_packed([t["x"], t["x"]], *layer, outs=list(o)), [narrow(), narrow()]),
        (lambda o: tp.gate_up(t["x"], *two, out=o), [narrow()]),
        (lambda o: tp.adapters(t["x"], *layer, *set_, out=o), [narrow()]),
        (lambda x, y, z: tp.adapters_backward(narrow(), t["x"], *layer, *set_, dx=x, da=y, db=z),
         [wide(), draw(2, 4, K), draw(2, N, 4)]),
        (lambda o: tp.gated(t["x"], *two, out=o), [narrow()]),
        (lambda x, y, z: tp.gated_backward(narrow(), gate, gate, *two, dx=x, dgate=y, dup=z), [wide(), narrow(), narrow()]),
        (lambda o: tp.loss_backward(torch.ones(M), wide(), out=o), [wide()]),
        (lambda o: tp.embed(t["tokens"], *layer[:2], K, BITS, extra=t["extra"], out=o), [wide()]),
        (lambda o: tp.embed_backward(wide(), t["tokens"], N, COUNT, dextra=o), [small()]),
    ]
    for i, (call, outs) in enumerate(calls):
        before = [o._version for o in outs]
        call(*outs)
        assert all(o._version > v for o, v in zip(outs, before)), i
    with torch.inference_mode():  # (such tensors have no counter)
        out = torch.empty(M, N, dtype=torch.bfloat16)
        assert tp.adapters(t["x"], *layer, *set_, out=out) is out


@pytest.mark.parametrize("what", ["adapters", "gated", "cross_entropy", "distill", "embed"])
def test_a_refused_capture_names_the_calls_to_make(monkeypatch, what):
    import re

    from trellis_coded_bit_prefill_amd import _autograd

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(ValueError, match=f"{what}.. is not differentiated") as refused:
        _autograd.refuse_capture(what)
    named = [f for f in re.findall(r"(\w+)\(\)", str(refused.value)) if f != "no_grad"]
    assert what in named and any(f.endswith("_backward") for f in named) and all(hasattr(tp, f) for f in named)


def embed(t, extra, **kw):
    return tp.embed(t["tokens"], t["codes"], t["scales"], K, BITS, extra=extra, **kw)


def test_embedding_gradients(plain):
    extra, dout = leaf(plain["extra"]), draw(M, K, seed=4)
    embed(plain, extra, scale=3.0).backward(dout)
    assert torch.equal(extra.grad, tp.embed_backward(dout, plain["tokens"], N, COUNT, scale=3.0))


def test_the_gradient_of_no_trained_rows(plain):
    """extra [0, K]: accepted forward, an empty gradient backward."""
    extra = leaf(plain["extra"][:0])
    out = embed(plain, extra)
    assert torch.equal(out, embed(plain, None)) and out.requires_grad
    out.sum().backward()
    assert extra.grad.shape == (0, K) and extra.grad.dtype == torch.bfloat16
