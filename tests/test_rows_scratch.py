"""Scratch memory of every kernel of the fine-tuned layers, from the compiler's
own report (gfx950): none, but for the few whose comments name it, at most what
they say. Compiling takes about a minute on the CPU."""
import os
import re
import subprocess

import pytest

from trellis_coded_bit_prefill_amd import _build

# bytes a lane: dense_kernel<column tiles, gated, transposed>, product_kernel<bits, transposed, six row tiles, ...>
STATED = {"dense_kernelILi6ELb0ELb0E": 16, "dense_kernelILi7ELb0ELb0E": 176, "dense_kernelILi8ELb0ELb0E": 312,
          "product_kernelILi2ELi2ELi6E": 48, "product_kernelILi3ELi2ELi6E": 48, "product_kernelILi4ELi2ELi6E": 48}


@pytest.mark.skipif(not os.path.exists(_build.hipcc()), reason="hipcc not available")
def test_scratch_is_what_the_comments_state(tmp_path):
    out = str(tmp_path / "rows.s")
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([_build.hipcc(), *flags, "--cuda-device-only", "-S", "-I", os.path.join(_build.ROOT, "include"),
                    "-o", out, *_build.ROWS_SOURCES], check=True, capture_output=True)
    with open(out) as f:
        report = re.findall(r"\.amdhsa_kernel (\S+)\n.*?\.amdhsa_private_segment_fixed_size (\d+)", f.read(), re.S)
    assert len(report) > 60
    for name, size in report:
        stated = next((v for k, v in STATED.items() if k in name), 0)
        assert int(size) <= stated, f"{name}: {size} bytes of scratch"
