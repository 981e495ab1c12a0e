"""Rules of the fine-tuned layers' planning code (tests/sanitize/rows_rules.hip),
on the CPU. The host side alone is compiled, so the device image that it would
register is left unresolved; no kernel is launched."""
import os

import pytest

from tests.test_sanitizers import HERE, ROOT, SAN_ENV, run


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    if not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not installed")
    exe = str(tmp_path_factory.mktemp("rules") / "rows_rules")
    run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17",
         "-ffp-contract=off", "-Wno-unused-command-line-argument", "-Wl,--unresolved-symbols=ignore-all",
         "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "trellis_coded_bit_prefill_amd", "csrc"),
         "-o", exe, os.path.join(HERE, "rows_rules.hip")], env=dict(os.environ))
    return run([exe], env=SAN_ENV).stdout


def test_slabs_are_whole_workgroup_tiles(rules):
    assert "slabs ok" in rules


def test_splits_are_near_the_fastest_measured(rules):
    assert "splits ok" in rules


def test_the_faster_measured_side_is_taken(rules):
    assert "sides ok" in rules
