"""What the fine-tuned layers' calls return and leave behind when the HIP
runtime refuses an allocation, a launch or a query: tests/sanitize/rows_space.hip
runs their host code over a stand-in for the runtime, on the CPU. The host side
alone is compiled, so the device image that it would register is left
unresolved.
"""
import os

import pytest

from tests.test_sanitizers import HERE, ROOT, SAN_ENV, run


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_errors_of_the_runtime(tmp_path):
    exe = str(tmp_path / "rows_space")
    run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17",
         "-ffp-contract=off", "-Wno-unused-command-line-argument", "-Wl,--unresolved-symbols=ignore-all",
         "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "trellis_coded_bit_prefill_amd", "csrc"),
         "-o", exe, os.path.join(HERE, "rows_space.hip")], env=dict(os.environ))
    assert "rows space ok" in run([exe], env=SAN_ENV).stdout
