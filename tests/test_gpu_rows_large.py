"""The fine-tuned layers where element offsets pass 32 bits: the same rows in a
large call and in a call of their own.

The sums of the two calls may be split differently, so an output may differ by
one bf16 step (2^-7 of it) and by the float32 sums' noise. With random terms of
size s, a sum of L of them is off by about 4 L s 2^-24 (L roundings of partial
sums of up to 4 sqrt(L) s, whose signs vary): 2^-16 at most for L = 256, 5e-4
for u (L = 17408, s = 0.12), and 4 sqrt(40) times that, 8 * 2^-9, for the 40
rows summed in da.
"""
import pytest

import trellis_coded_bit_prefill_amd as tp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GiB")
    tp.load_library()
    yield
    torch.cuda.empty_cache()


def layer(g, n, k, bits):
    import torch

    codes = torch.randint(-2**31, 2**31 - 1, (n, k * bits // 32), generator=g, device="cuda", dtype=torch.int32)
    return codes, (torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005).to(torch.bfloat16)


def normal(g, *shape):
    import torch

    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return t.normal_(generator=g)


def close(got, want):
    off = (got.float() - want.float()).abs()
    return bool((off <= want.float().abs() * 2.0 ** -7 + 2.0 ** -9).all())


def test_outputs_past_32_bits():
    import torch

    m, n, k, bits, rank = 140000, 17408, 256, 2, 5
    assert m * n > 2**31
    print(f"large m={m} n={n}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(51)
    codes, scales = layer(g, n, k, bits)
    x, dout = normal(g, m, k), normal(g, m, n)
    a, b = normal(g, 2, rank, k) * 0.06, normal(g, 2, n, rank) * 0.06
    gain = torch.tensor([0.5, 2.0], device="cuda")
    # adapters in the first and in the last rows only
    index = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    index[:40] = 1
    index[m - 40:] = 0
    rows = torch.cat([torch.arange(64), torch.arange(2**31 // n - 32, 2**31 // n + 32), torch.arange(m - 64, m)]).cuda()
    out = tp.adapters(x, codes, scales, bits, a, b, gain, index)
    few = (x[rows].contiguous(), codes, scales, bits, a, b, gain, index[rows].contiguous())
    assert close(out[rows], tp.adapters(*few))
    del out
    dx, da, db = tp.adapters_backward(dout, x, codes, scales, bits, a, b, gain, index)
    fx, fa, fb = tp.adapters_backward(dout[rows].contiguous(), *few)
    assert close(dx[rows], fx) and close(da / 8, fa / 8) and close(db, fb)
    del dx, dout
    h, gate, up = tp.gated(x, codes, scales, codes, scales, bits, keep=True)
    want = tp.gated(few[0], codes, scales, codes, scales, bits, keep=True)
    for got, w in zip((h, gate, up), want):
        assert close(got[rows], w)
    torch.cuda.synchronize()


def test_factors_past_32_bits():
    import torch

    m, n, k, bits, rank, count = 3, 1 << 22, 256, 2, 128, 5
    assert count * n * rank > 2**31
    print(f"large factors n={n} rank={rank} count={count}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(52)
    codes, scales = layer(g, n, k, bits)
    x, dout = normal(g, m, k), normal(g, m, n)
    a, b = normal(g, count, rank, k) * 0.06, normal(g, count, n, rank)
    gain = torch.full((count,), 0.01, device="cuda")
    index = torch.tensor([4, -1, 4], dtype=torch.int32, device="cuda")
    one = (a[4:].contiguous(), b[4:].contiguous(), gain[4:].contiguous(), torch.where(index < 0, -1, 0).to(torch.int32))
    assert close(tp.adapters(x, codes, scales, bits, a, b, gain, index), tp.adapters(x, codes, scales, bits, *one))
    dx, da, db = tp.adapters_backward(dout, x, codes, scales, bits, a, b, gain, index)
    ex, ea, eb = tp.adapters_backward(dout, x, codes, scales, bits, *one)
    # the same sums in the same order: the products differ in nothing but the factors' place
    assert torch.equal(dx, ex) and torch.equal(da[4:], ea) and torch.equal(db[4:], eb)
    assert not bool(da[:4].any()) and not bool(db[:4].any())
    torch.cuda.synchronize()
