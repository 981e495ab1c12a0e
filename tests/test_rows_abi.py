"""Refusals of the fine-tuned layers' entry points, on the CPU: every
out-of-domain call is rejected before any GPU work."""
import pytest

import trellis_coded_bit_prefill_amd as tp

FAKE = 1 << 20  # a 16-byte aligned address that is never dereferenced
GOOD = dict(n=260, k=512, bits=4)


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(tp.LIB_PATH):
        from trellis_coded_bit_prefill_amd import _build

        _build.build()
    return tp.load_library()


ADAPTERS = ["x", "m", "codes", "scales", "g", "a", "b", "gain", "index", "count", "rank", "out"]
BACKWARD = ["dout", "x", "m", "codes", "scales", "g", "a", "b", "gain", "index", "count", "rank", "dx", "da", "db"]
GATED = ["x", "m", "codes_gate", "scales_gate", "codes_up", "scales_up", "g", "h", "gate", "up"]
GATED_BACKWARD = ["dh", "gate", "up", "m", "codes_gate", "scales_gate", "codes_up", "scales_up", "g", "dx", "dgate",
                  "dup"]
ENTRIES = {"trellis_adapters": ADAPTERS, "trellis_adapters_backward": BACKWARD, "trellis_gated": GATED,
           "trellis_gated_backward": GATED_BACKWARD}


def call(lib, entry, **change):
    args = []
    for name in ENTRIES[entry]:
        value = {"m": 7, "g": tp.geom(**GOOD), "count": 2, "rank": 8}.get(name, FAKE)
        args.append(change.get(name, value))
    return getattr(lib, entry)(*args, None)


@pytest.mark.parametrize("entry", list(ENTRIES))
def test_refusals(lib, entry):
    for g in (tp.geom(260, 500, 4), tp.geom(258, 512, 4), tp.geom(260, 512, 5), tp.geom(260, 512, 4, 128),
              tp.geom(260, 512, 4, 256, 16), tp.geom(0, 512, 4), tp.geom(260, 0, 4)):
        assert call(lib, entry, g=g) == tp.E_GEOMETRY
    for m in (0, -1, tp.MAX_ROWS + 1, -2**31):
        assert call(lib, entry, m=m) == tp.E_M
    for name in ENTRIES[entry]:
        if name in ("m", "g", "count", "rank"):
            continue
        if not (entry == "trellis_gated" and name in ("gate", "up")):
            assert call(lib, entry, **{name: None}) == tp.E_NULL, name
        assert call(lib, entry, **{name: FAKE + 1}) == tp.E_ALIGN, name
        if not name.startswith("scales"):
            assert call(lib, entry, **{name: FAKE + 2}) == tp.E_ALIGN, name
    # geometry first, then m, then pointers
    assert call(lib, entry, g=tp.geom(260, 500, 4), m=0) == tp.E_GEOMETRY
    assert call(lib, entry, m=0, **{ENTRIES[entry][0]: None}) == tp.E_M


@pytest.mark.parametrize("entry", ["trellis_adapters", "trellis_adapters_backward"])
def test_adapter_refusals(lib, entry):
    for change in ({"count": 0}, {"count": -1}, {"count": tp.MAX_ADAPTERS + 1}, {"rank": 0}, {"rank": -3},
                   {"rank": tp.MAX_RANK + 1}):
        assert call(lib, entry, **change) == tp.E_ADAPTERS
    assert "rank" in tp.status_string(tp.E_ADAPTERS)
    with pytest.raises(ValueError):
        tp.adapters_raw(FAKE, 1, FAKE, FAKE, tp.geom(**GOOD), FAKE, FAKE, FAKE, FAKE, 1, 129, FAKE, 0)


def test_path_hook_checks_its_arguments(lib):
    tp.force_path(True, 16)
    tp.force_path(False)
    tp.force_path(None)
    assert lib.trellis_test_force_path(2, 0) == -2
    assert lib.trellis_test_force_path(0, -1) == -2
    with pytest.raises(ValueError):
        tp.force_path(5)


def test_python_checks_refuse_host_tensors():
    import torch

    x = torch.zeros((3, 512), dtype=torch.bfloat16)
    codes = torch.zeros((260, 64), dtype=torch.int32)
    scales = torch.zeros(260, dtype=torch.bfloat16)
    a, b = torch.zeros((2, 8, 512), dtype=torch.bfloat16), torch.zeros((2, 260, 8), dtype=torch.bfloat16)
    gain, index = torch.zeros(2), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        tp.adapters(x, codes, scales, 4, a, b, gain, index)
    with pytest.raises(ValueError, match="device"):
        tp.adapters_backward(x, x, codes, scales, 4, a, b, gain, index)
    with pytest.raises(ValueError, match="device"):
        tp.gated(x, codes, scales, codes, scales, 4)
    with pytest.raises(ValueError, match="device"):
        tp.gated_backward(x, x, x, codes, scales, codes, scales, 4)
    with pytest.raises(TypeError):
        tp.adapters(x.float(), codes, scales, 4, a, b, gain, index)
