"""Layouts of the losses over a sweep of sizes, on the CPU. The host side alone is
compiled, so the device image that it would register is left unresolved; no
kernel is launched."""
import os

import pytest

from tests.test_sanitizers import HERE, ROOT, SAN_ENV, run


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not installed")
    exe = str(tmp_path_factory.mktemp("plan") / "vocabulary_plan")
    run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17",
         "-ffp-contract=off", "-Wno-unused-command-line-argument", "-Wl,--unresolved-symbols=ignore-all",
         "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "trellis_coded_bit_prefill_amd", "csrc"),
         "-o", exe, os.path.join(HERE, "vocabulary_plan.hip")], env=dict(os.environ))
    return run([exe], env=SAN_ENV).stdout


def test_layouts_of_all_sizes(plan):
    assert "vocabulary plan ok" in plan


def test_the_faster_measured_side_is_taken(plan):
    assert "vocabulary sides ok" in plan
