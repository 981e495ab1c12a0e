"""distill()'s lists on the GPU, on all paths: logits of any float32 value."""
import numpy as np
import pytest

import trellis_coded_bit_prefill_amd as tp
from tests import vocabulary_reference as ref
from tests.helpers import to_dev_bf16
from tests.test_gpu_loss import check_all, dev, need_gpu, packed, path  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min


def check(what, d, t, got, want):
    """check_all() with float32's range: at T = 0.01 a row's only entry is so likely that its loss and all p are below
    the smallest normal float32, 2^-126, where the hardware's exponential gives 0 and the reference's bounds, being
    relative, go on falling. An exponential is then off by up to 2^-126, and so is the loss, before the factor T^2 and
    again as a result: (1 + T^2) 2^-126. Each of N terms of dx is off by as much, times T |W|, in the exponential,
    in the operand and in the term itself: 3 N (1 + T) 2^-126 max|W|."""
    tiny = 2.0 ** -126
    floor = {"loss": (1 + t * t) * tiny, "lse": 0.0,
             "dx": 3 * len(d["w"]) * (1 + t) * tiny * max(1.0, np.abs(d["w"]).max())}
    check_all(what, got, {k: (value, bound + floor[k]) for k, (value, bound) in want.items()})


def distill(d, index, logits, t):
    return tp.distill(to_dev_bf16(d["x_bits"]), *packed(d), dev(index), dev(logits), temperature=t, keep=True)


@pytest.mark.parametrize("top,t", [(1, 1.0), (1, 0.01), (4, 1.0), (4, 0.01), (70, 2.0)])
@pytest.mark.parametrize("m,n", [(5, 260), (3, 20004), (300, 260)])
def test_teachers_of_the_largest_and_lowest_logits(path, m, n, top, t):  # noqa: F811
    """Finite logits that float32 cannot hold once they are scaled by 1 / T: only their differences count."""
    import torch

    print(f"largest logits {m} {n} top {top} T {t} {path}", flush=True)
    d = ref.draw(np.random.default_rng(m + n + top), m, n, 256, 4, top=top)
    even = distill(d, d["index"], np.zeros((m, top), np.float32), t)
    check("even", d, t, even, ref.loss(d, d["index"], np.zeros((m, top), np.float32), t))
    for z in (LOWEST, -LOWEST, np.float32(-3e36), np.float32(3e38)):
        got = distill(d, d["index"], np.full((m, top), z, np.float32), t)
        assert all(torch.equal(a, b) for a, b in zip(got, even)), z
    # an entry that a mask of the type's lowest value hides: probability 0, but not none
    logits = d["logits"].copy()
    logits[:, 1::2] = LOWEST
    check("masked", d, t, distill(d, d["index"], logits, t), ref.loss(d, d["index"], logits, t))
