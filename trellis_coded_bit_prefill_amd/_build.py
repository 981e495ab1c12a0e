"""Compile the HIP library ``libtrellis.so`` for gfx950 with hipcc."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libtrellis.so")
SOURCES = [os.path.join(PKG, "csrc", "trellis.hip")]       # the narrow-batch layer
ROWS_SOURCES = [os.path.join(PKG, "csrc", "rows.hip")]     # fine-tuned layers, any number of rows

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # exact decode arithmetic: no multiply-add contraction
    "-ffp-contract=off",
    # no packed-fp32 VALU instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(verbose: bool = False) -> str:
    """Always recompiles (the sources side by side); writes the library
    atomically next to this file."""
    tmp = LIB + ".tmp%d" % os.getpid()

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)

    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES + ROWS_SOURCES]
        cmds = [[hipcc(), *compile_flags, "-I", os.path.join(ROOT, "include"), "-c", "-o", o, s]
                for o, s in zip(objects, SOURCES + ROWS_SOURCES)]
        with concurrent.futures.ThreadPoolExecutor(len(cmds)) as pool:
            list(pool.map(run, cmds))
        run([hipcc(), *HIPCC_FLAGS, "-o", tmp, *objects])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
