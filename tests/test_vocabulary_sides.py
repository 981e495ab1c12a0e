"""The rule between the losses' two ways against measured times of long lists and
of matrices that it was not fitted to, on the CPU. The host side alone is
compiled, so the device image that it would register is left unresolved; no
kernel is launched."""
import os

import pytest

from tests.test_sanitizers import HERE, ROOT, SAN_ENV, run


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_the_faster_measured_side_is_taken(tmp_path):
    exe = str(tmp_path / "vocabulary_sides")
    run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17",
         "-ffp-contract=off", "-Wno-unused-command-line-argument", "-Wl,--unresolved-symbols=ignore-all",
         "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "trellis_coded_bit_prefill_amd", "csrc"),
         "-o", exe, os.path.join(HERE, "vocabulary_sides.hip")], env=dict(os.environ))
    assert "sides ok" in run([exe], env=SAN_ENV).stdout
