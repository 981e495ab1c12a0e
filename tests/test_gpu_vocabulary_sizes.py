"""The losses and the embedding at the largest accepted vocabulary (2^22 rows) and
width (2^18 columns), against the formulas in float64 on the GPU."""
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests.test_gpu_vocabulary_run import need_gpu, plain_loss  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


def matrix(g, n, k, bits):
    import torch

    codes = torch.randint(-2**31, 2**31, (n, k * bits // 32), generator=g, device="cuda", dtype=torch.int32)
    return codes, (torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005).bfloat16()


@pytest.mark.parametrize("path", [False, True], ids=["few", "many"])
@pytest.mark.parametrize("m,n,k,bits", [(2, 1 << 22, 256, 2), (40, 68, 1 << 18, 4), (300, 68, 1 << 18, 3)])
def test_losses(m, n, k, bits, path):
    """x has 64 numbers a row other than zero, spread over all columns: a logit is a float32 sum of 64 products. Bounds
    as in test_chunks_of_rows (tests/test_gpu_vocabulary_run.py)."""
    import torch

    print(f"loss {m} {n} {k} {bits} {path}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + k)
    codes, scales = matrix(g, n, k, bits)
    x = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16)
    at = (torch.arange(64, device="cuda") * (k // 64) + torch.randint(0, k // 64, (m, 64), generator=g, device="cuda"))
    x.scatter_(1, at, (torch.randn(m, 64, generator=g, device="cuda") * 10).bfloat16())
    target = torch.randint(0, n, (m,), generator=g, device="cuda", dtype=torch.int32)
    target[0] = n - 1
    try:
        tp.force_path(path)
        got = tp.cross_entropy(x, codes, scales, bits, target, keep=True)
        short = tp.cross_entropy(x, codes, scales, bits, target)
    finally:
        tp.force_path(None)
    w = tp.decode(codes, scales, k, bits)
    loss, lse, dx = plain_loss(x, w, target, torch.float64)
    largest = w.abs().max().double()
    el = 64 * E24 * (x.double().abs().sum(1) * largest) + 4 * E24 * 40
    bound = 2 * el + 2.0 ** -17 + 8 * E24 * lse.abs()
    for o in (got, short):
        assert ((o[0] - loss).abs() <= 2 * bound).all() and ((o[1] - lse).abs() <= bound).all()
    off = (got[2].double() - dx).abs()
    assert (off <= 2 * largest * (2 * 2.0 ** -8 + 2 * bound[:, None]) + 2.0 ** -8 * dx.abs()).all()
    assert (off.norm(dim=1) <= 2.0 ** -7 * dx.norm(dim=1) + 1e-6).all()


@pytest.mark.parametrize("m,n,k,count", [(5, 1 << 22, 256, 3), (40, 68, 1 << 18, 5), (700, 8, 1 << 18, 1)])
def test_embedding(m, n, k, count):
    import torch

    print(f"embed {m} {n} {k} {count}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n)
    codes, scales = matrix(g, n, k, 2)
    extra = torch.randn(count, k, generator=g, device="cuda").bfloat16()
    tokens = torch.randint(0, n + count, (m,), generator=g, device="cuda", dtype=torch.int32)
    tokens[:5] = torch.tensor([n - 1, n, n + count - 1, n + count, 0])
    table = torch.cat([tp.decode(codes, scales, k, 2), extra, torch.zeros_like(extra[:1])])
    assert torch.equal(tp.embed(tokens, codes, scales, k, 2, extra=extra), table[tokens.long()])
    # small whole numbers: every float32 sum is exact, whatever its order
    dout = torch.randint(-2, 3, (m, k), generator=g, device="cuda").bfloat16()
    t = tokens.long() - n
    at = ((t >= 0) & (t < count)).nonzero()[:, 0]
    want = torch.zeros(count, k, device="cuda").index_add_(0, t[at], dout[at].float())
    assert torch.equal(tp.embed_backward(dout, tokens, n, count), want.bfloat16())


def test_gradients_of_64_gib():
    """2^20 rows of 32768 columns, in place: 2^32 vectors of 16 bytes, several a thread."""
    import torch

    print("loss_backward 64 GiB", flush=True)
    m, k = 1 << 20, 32768
    dx = torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
    columns = (torch.arange(k, device="cuda") % 5 - 2).bfloat16()
    dx.copy_(columns)
    dloss = (torch.arange(m, device="cuda") % 61).float()
    assert tp.loss_backward(dloss, dx, out=dx) is dx
    for r0 in range(0, m, 1 << 16):
        r = slice(r0, r0 + (1 << 16))
        assert torch.equal(dx[r], dloss[r, None].bfloat16() * columns)  # (whole numbers up to 122: exact)
    del dx
    torch.cuda.empty_cache()
