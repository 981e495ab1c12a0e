"""What autograd records for adapters() and gated(), on the CPU: the library's
four calls are replaced by the plain formulas in float64 on host tensors, so
what is tested is which call is recorded, what is handed to the backward calls
and where the gradients go."""
import ctypes

import pytest
import torch

import trellis_coded_bit_prefill_amd as tp

M, N, K, BITS, RANK, COUNT = 6, 8, 256, 2, 3, 2


def silu_parts(gate):
    s = torch.sigmoid(gate)
    return gate * s, s * (1 + gate * (1 - s))


@pytest.fixture
def plain(monkeypatch):
    """The calls' inputs, and a record of the raw calls made."""
    g = torch.Generator().manual_seed(3)

    def draw(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    t = {"x": draw(M, K), "a": draw(COUNT, RANK, K), "b": draw(COUNT, N, RANK), "gain": torch.tensor([0.5, 2.0]),
         "index": torch.tensor([1, -1, 0, 0, 1, 5], dtype=torch.int32),
         "codes": torch.zeros((N, K * BITS // 32), dtype=torch.int32), "scales": draw(N), "w": draw(N, K), "w2": draw(N, K)}
    calls = []

    def put(address, value):
        value = value.to(torch.bfloat16).contiguous()
        ctypes.memmove(address, value.data_ptr(), value.numel() * 2)

    def at(address, *shape):
        out = torch.empty(shape, dtype=torch.bfloat16)
        ctypes.memmove(out.data_ptr(), address, out.numel() * 2)
        return out.double()

    def part():
        own = t["index"][:, None] == torch.arange(COUNT)
        return (own * t["gain"]).double()

    def adapters_raw(x, m, codes, scales, geom, a, b, gain, index, count, rank, out, stream):
        calls.append("adapters")
        x, a, b = at(x, M, K), at(a, COUNT, RANK, K), at(b, COUNT, N, RANK)
        low = sum(part()[:, i:i + 1] * (x @ a[i].T @ b[i].T) for i in range(COUNT))
        put(out, x @ t["w"].double().T + low)

    def adapters_backward_raw(dout, x, m, codes, scales, geom, a, b, gain, index, count, rank, dx, da, db, stream):
        calls.append("adapters_backward")
        assert dout % 16 == 0
        dout, x, a, b, p = at(dout, M, N), at(x, M, K), at(a, COUNT, RANK, K), at(b, COUNT, N, RANK), part()
        put(dx, dout @ t["w"].double() + sum(p[:, i:i + 1] * (dout @ b[i] @ a[i]) for i in range(COUNT)))
        put(da, torch.stack([(p[:, i:i + 1] * dout @ b[i]).T @ x for i in range(COUNT)]))
        put(db, torch.stack([dout.T @ (p[:, i:i + 1] * x @ a[i].T) for i in range(COUNT)]))

    def gated_raw(x, m, cg, sg, cu, su, geom, h, gate, up, stream):
        calls.append("gated keep" if gate else "gated")
        g, u = at(x, M, K) @ t["w"].double().T, at(x, M, K) @ t["w2"].double().T
        put(h, silu_parts(g)[0] * u)
        if gate:
            put(gate, g)
            put(up, u)

    def gated_backward_raw(dh, gate, up, m, cg, sg, cu, su, geom, dx, dgate, dup, stream):
        calls.append("gated_backward")
        assert dh % 16 == 0
        dh, g, u = at(dh, M, N), at(gate, M, N), at(up, M, N)
        silu, slope = silu_parts(g)
        put(dgate, dh * u * slope)
        put(dup, dh * silu)
        put(dx, dh * u * slope @ t["w"].double() + dh * silu @ t["w2"].double())

    for f in (adapters_raw, adapters_backward_raw, gated_raw, gated_backward_raw):
        monkeypatch.setattr(tp, f.__name__, f)
    monkeypatch.setattr(tp, "_stream_handle", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    check = tp._check_tensor
    monkeypatch.setattr(tp, "_check_tensor", lambda name, v, *r: check(name, v, *r) if not isinstance(v, torch.Tensor) else None)
    return t, calls


def adapters(t, **change):
    s = {**t, **change}
    return tp.adapters(s["x"], s["codes"], s["scales"], BITS, s["a"], s["b"], s["gain"], s["index"],
                       **({"out": s["out"]} if "out" in s else {}))


def gated(t, **change):
    s = {**t, **change}
    return tp.gated(s["x"], s["codes"], s["scales"], s["codes"], s.get("scales2", s["scales"]), BITS,
                    **{k: s[k] for k in ("out", "keep") if k in s})


def leaf(v):
    return v.clone().requires_grad_()


def test_adapters_gradients(plain):
    t, calls = plain
    x, a, b = leaf(t["x"]), leaf(t["a"]), leaf(t["b"])
    out = adapters(t, x=x, a=a, b=b)
    assert torch.equal(out, adapters(t))
    dout = torch.randn(M, N).to(torch.bfloat16)
    out.backward(dout)
    want = tp.adapters_backward(dout, t["x"], t["codes"], t["scales"], BITS, t["a"], t["b"], t["gain"], t["index"])
    assert all(torch.equal(p.grad, w) for p, w in zip((x, a, b), want))
    assert calls == ["adapters", "adapters", "adapters_backward", "adapters_backward"]


@pytest.mark.parametrize("name", ["x", "a", "b"])
def test_one_input_alone(plain, name):
    t, _ = plain
    v = leaf(t[name])
    # an expanded gradient, as sum() hands it over
    adapters(t, **{name: v}).sum().backward()
    ones = torch.ones(M, N, dtype=torch.bfloat16)
    want = tp.adapters_backward(ones, t["x"], t["codes"], t["scales"], BITS, t["a"], t["b"], t["gain"], t["index"])
    assert torch.equal(v.grad, want["xab".index(name)])


def test_a_gradient_that_is_a_slice(plain):
    t, _ = plain
    whole = torch.randn(M * N + 4).to(torch.bfloat16)
    dout = next(v for v in (whole[i:i + M * N].view(M, N) for i in range(5)) if v.data_ptr() % 16)
    x = leaf(t["x"])
    adapters(t, x=x).backward(dout)
    gated(t, x=x).backward(dout)


@pytest.mark.parametrize("keep", [False, True])
def test_gated_gradients(plain, keep):
    t, calls = plain
    x = leaf(t["x"])
    got = gated(t, x=x, keep=keep)
    want = gated(t, keep=True)
    h = got[0] if keep else got
    assert torch.equal(h, want[0]) and (not keep or all(torch.equal(p, q) for p, q in zip(got, want)))
    dh = torch.randn(M, N).to(torch.bfloat16)
    h.backward(dh)
    assert torch.equal(x.grad, tp.gated_backward(dh, *want[1:], t["codes"], t["scales"], t["codes"], t["scales"], BITS)[0])


def test_a_gradient_of_the_kept_projections_is_refused(plain):
    t, _ = plain
    h, gate, up = gated(t, x=leaf(t["x"]), keep=True)
    with pytest.raises(RuntimeError, match="kept projections"):
        (h.float().sum() + up.float().sum()).backward()


def test_a_run_of_both(plain):
    t, calls = plain
    down = {**t, "codes": torch.zeros((N, 256 * BITS // 32), dtype=torch.int32)}
    x, a = leaf(t["x"]), leaf(t["a"])
    h = gated(t, x=x)
    y = adapters(down, x=torch.nn.functional.pad(h, (0, K - N)), a=a)
    y.float().square().sum().backward()
    assert bool(x.grad.any()) and bool(a.grad.any())
    assert calls == ["gated keep", "adapters", "adapters_backward", "gated_backward"]


def test_what_is_not_recorded(plain):
    t, calls = plain
    x = leaf(t["x"])
    with torch.no_grad():
        assert adapters(t, x=x, out=torch.empty(M, N, dtype=torch.bfloat16)).grad_fn is None
        assert gated(t, x=x).grad_fn is None
    with torch.inference_mode():
        assert not gated(t).requires_grad
    assert not adapters(t).requires_grad and not gated(t, keep=True)[1].requires_grad
    assert calls.count("gated") == 2


def test_refusals(plain):
    t, calls = plain
    x = leaf(t["x"])
    out = torch.empty(M, N, dtype=torch.bfloat16)
    for call in (adapters, gated):
        with pytest.raises(ValueError, match="out="):
            call(t, x=x, out=out)
    with pytest.raises(ValueError, match="gain gets no gradient"):
        adapters(t, gain=leaf(t["gain"]))
    with pytest.raises(ValueError, match="scales gets no gradient"):
        adapters(t, x=x, scales=leaf(t["scales"]))
    with pytest.raises(ValueError, match="scales_up gets no gradient"):
        gated(t, scales2=leaf(t["scales"]))
    import torch.autograd.forward_ad as forward_ad

    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t["x"], torch.ones_like(t["x"]))
        for call in (adapters, gated):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call(t, x=dual)
        calls.clear()
        adapters(t)
    assert calls == ["adapters"]


def test_a_second_derivative_is_refused(plain):
    t, _ = plain
    for call in (adapters, gated):
        x = leaf(t["x"])
        grad, = torch.autograd.grad(call(t, x=x).float().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            grad.float().sum().backward()


def test_a_changed_input_is_noticed(plain):
    t, _ = plain
    x, index = leaf(t["x"]), t["index"].clone()
    out = adapters(t, x=x, index=index)
    index.fill_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_capture_is_refused(plain, monkeypatch):
    t, calls = plain
    x = leaf(t["x"])
    outs = adapters(t, x=x), gated(t, x=x)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    calls.clear()
    for call in (adapters, gated):
        with pytest.raises(ValueError, match="captured"):
            call(t, x=x)
        with torch.no_grad():
            call(t, x=x)
    assert calls == ["adapters", "gated"]
    for out in outs:
        with pytest.raises(ValueError, match="captured"):
            out.sum().backward()
