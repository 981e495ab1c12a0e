"""Register use of the fine-tuned layers' kernels, from the compiler's own
report and device assembly (gfx950): the loops that do the work must not touch
scratch memory, which is HBM, and the copies to LDS, written as inline assembly
that the compiler's hazard recognizer does not look into, must carry the wait
states that they need. Compiling takes about a minute on the CPU."""
import os
import re
import subprocess

import pytest

from trellis_coded_bit_prefill_amd import _build

needs_hipcc = pytest.mark.skipif(not os.path.exists(_build.hipcc()), reason="hipcc not available")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "rows.s")
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([_build.hipcc(), *flags, "--cuda-device-only", "-S", "-I", os.path.join(_build.ROOT, "include"),
                    "-o", out, *_build.ROWS_SOURCES], check=True, capture_output=True)
    with open(out) as f:
        blocks = re.split(r"\n(?=_Z\S*:)", f.read())
    return {b.split(":", 1)[0]: b for b in blocks if b.startswith("_Z")}


def basic_blocks(blk):
    out, cur = [], []
    for line in blk.split("\n"):
        t = line.strip()
        if re.match(r"^(\.LBB\S+|; %bb\.\d+):", t):
            cur = []
            out.append(cur)
        elif t and not t.startswith((".", ";")):
            cur.append(t.split()[0])
    return out


@needs_hipcc
def test_multiplying_loops_use_no_scratch(kernels):
    seen = {"product_kernel": 0, "dense_kernel": 0}
    for name, blk in kernels.items():
        kind = next((k for k in seen if k in name), None)
        if kind is None:
            continue
        loops = [b for b in basic_blocks(blk)
                 if b.count("v_mfma_f32_16x16x32_bf16") >= 4 and (b.count("ds_read_b128") >= 1)]
        assert loops, f"{name}: no multiplying block found"
        for b in loops:
            assert not any(m.startswith("scratch_") for m in b), f"{name} spills in its loop"
        seen[kind] += 1
    # 3 bit widths x (forward and gated: 5 row tiles, transposed: 4); column tiles x directions
    assert seen == {"product_kernel": 42, "dense_kernel": 13}


@needs_hipcc
def test_copies_to_lds_carry_their_wait_states(kernels):
    seen = 0
    for name, blk in kernels.items():
        lines = [l.strip() for l in blk.split("\n") if l.strip() and not l.strip().startswith((";", "."))]
        for i, line in enumerate(lines):
            if line.startswith("global_load_lds_dwordx4"):
                assert lines[i - 1] == "s_nop 4" and lines[i - 2].startswith("s_mov_b32 m0"), f"{name}: {line}"
                seen += 1
    assert seen > 0


@needs_hipcc
def test_no_packed_float32_arithmetic(kernels):
    for name, blk in kernels.items():
        assert not re.search(r"v_pk_(add|mul|fma)_f32", blk), name
