"""AddressSanitizer / UndefinedBehaviorSanitizer build of the fine-tuned layers'
host code (validation, planning, workspace bookkeeping), driven through every
entry point by tests/sanitize/rows_driver.cpp on the CPU: the sanitizers are on
for the host compilation only, device code never runs here, and with no GPU
present the in-domain calls must return TRELLIS_E_HIP.
"""
import os

import pytest

from tests.test_sanitizers import HERE, ROOT, SAN_ENV, run


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="checks the no-GPU error path; a GPU is present")
def test_rows_host_side_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "rows_driver")
    env = dict(os.environ)
    env.pop("HIP_VISIBLE_DEVICES", None)
    run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-ffp-contract=off",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument",
         "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
         "-Xarch_host", "-fno-sanitize-recover=undefined",
         "-I", os.path.join(ROOT, "include"), "-o", exe, os.path.join(HERE, "rows_driver.cpp"),
         os.path.join(ROOT, "trellis_coded_bit_prefill_amd", "csrc", "rows.hip")], env=env)
    r = run([exe], env=dict(SAN_ENV, HIP_VISIBLE_DEVICES=""))
    assert "rows driver ok" in r.stdout


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_layouts_of_all_sizes_under_ubsan(tmp_path):
    exe = str(tmp_path / "rows_plan")
    run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-ffp-contract=off",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument",
         "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "trellis_coded_bit_prefill_amd", "csrc"),
         "-o", exe, os.path.join(HERE, "rows_plan.hip")], env=dict(os.environ))
    assert "rows plan ok" in run([exe], env=SAN_ENV).stdout
