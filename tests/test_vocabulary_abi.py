"""Refusals of the losses' and the embedding's entry points, on the CPU: every
out-of-domain call is rejected before any GPU work."""
import os

import pytest

import trellis_coded_bit_prefill_amd as tp

FAKE = 1 << 20  # a 16-byte aligned address that is never dereferenced
GOOD = dict(n=260, k=512, bits=4)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tp.LIB_PATH):
        from trellis_coded_bit_prefill_amd import _build

        _build.build()
    return tp.load_library()


ENTRIES = {
    "trellis_cross_entropy": ["x", "m", "codes", "scales", "g", "target", "loss", "lse", "dx"],
    "trellis_distill": ["x", "m", "codes", "scales", "g", "index", "logits", "top", "temperature", "loss", "lse", "dx"],
    "trellis_loss_backward": ["dloss", "dx", "m", "k", "out"],
    "trellis_embed": ["tokens", "m", "codes", "scales", "g", "scale", "extra", "count", "out"],
    "trellis_embed_backward": ["dout", "tokens", "m", "k", "first", "count", "scale", "dextra"],
}
NUMBERS = {"m": 7, "k": 512, "top": 3, "temperature": 1.0, "count": 5, "first": 260, "scale": 1.0}
OPTIONAL = {"trellis_cross_entropy": ("dx",), "trellis_distill": ("dx",)}
WORDS = ("target", "index", "logits", "tokens", "loss", "lse", "dloss")  # 4-byte aligned


def call(lib, entry, **change):
    args = [change.get(name, tp.geom(**GOOD) if name == "g" else NUMBERS.get(name, FAKE)) for name in ENTRIES[entry]]
    return getattr(lib, entry)(*args, None)


@pytest.mark.parametrize("entry", list(ENTRIES))
def test_refusals(lib, entry):
    names = ENTRIES[entry]
    if "g" in names:
        for g in (tp.geom(260, 500, 4), tp.geom(258, 512, 4), tp.geom(260, 512, 5), tp.geom(260, 512, 4, 128),
                  tp.geom(260, 512, 4, 256, 16), tp.geom(0, 512, 4), tp.geom(260, 0, 4)):
            assert call(lib, entry, g=g) == tp.E_GEOMETRY
    else:
        for k in (0, -256, 255, 128, (1 << 18) + 256):
            assert call(lib, entry, k=k) == tp.E_GEOMETRY
    for m in (0, -1, tp.MAX_ROWS + 1, -2**31):
        assert call(lib, entry, m=m) == tp.E_M
    for name in names:
        if name in NUMBERS or name == "g":
            continue
        if name not in OPTIONAL.get(entry, ()):
            assert call(lib, entry, **{name: None}) == tp.E_NULL, name
        assert call(lib, entry, **{name: FAKE + 1}) == tp.E_ALIGN, name
        if name not in ("scales",):
            assert call(lib, entry, **{name: FAKE + 2}) == tp.E_ALIGN, name
        if name not in WORDS + ("scales",):
            assert call(lib, entry, **{name: FAKE + 8}) == tp.E_ALIGN, name
    # m before pointers
    assert call(lib, entry, m=0, **{names[0]: None}) == tp.E_M


def test_ranges(lib):
    for change in ({"top": 0}, {"top": -1}, {"top": tp.MAX_TOP + 1}, {"temperature": 0.0}, {"temperature": -1.0},
                   {"temperature": 0.0099}, {"temperature": 100.1}, {"temperature": float("nan")},
                   {"temperature": float("inf")}):
        assert call(lib, "trellis_distill", **change) == tp.E_RANGE, change
    for change in ({"count": -1}, {"count": tp.MAX_TRAINED + 1}, {"scale": float("nan")}, {"scale": float("-inf")}):
        assert call(lib, "trellis_embed", **change) == tp.E_RANGE, change
    for change in ({"count": 0}, {"count": tp.MAX_TRAINED + 1}, {"scale": float("inf")}, {"first": -1},
                   {"first": tp.MAX_N + 1}):
        assert call(lib, "trellis_embed_backward", **change) == tp.E_RANGE, change
    assert call(lib, "trellis_embed", extra=None) == tp.E_NULL
    assert "temperature" in tp.status_string(tp.E_RANGE)


def test_python_checks_refuse_host_tensors():
    import torch

    x = torch.zeros((3, 512), dtype=torch.bfloat16)
    codes, scales = torch.zeros((260, 64), dtype=torch.int32), torch.zeros(260, dtype=torch.bfloat16)
    t = torch.zeros(3, dtype=torch.int32)
    for call_ in (lambda: tp.cross_entropy(x, codes, scales, 4, t),
                  lambda: tp.distill(x, codes, scales, 4, t[:, None], torch.zeros(3, 1)),
                  lambda: tp.loss_backward(torch.zeros(3), x), lambda: tp.embed(t, codes, scales, 512, 4),
                  lambda: tp.embed_backward(x, t, 260, 2)):
        with pytest.raises(ValueError, match="device"):
            call_()
    with pytest.raises(TypeError):
        tp.cross_entropy(x.float(), codes, scales, 4, t)
    for tokens in (None, [0, 1], t.float()):
        with pytest.raises(TypeError):
            tp.embed(tokens, codes, scales, 512, 4)
