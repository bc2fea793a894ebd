"""Build libdopt.so (host mapper + gfx950 kernels) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SO = os.path.join(HERE, "libdopt.so")
SOURCES = [os.path.join(HERE, "csrc", "mapper.cpp"), os.path.join(HERE, "csrc", "step.hip"),
           os.path.join(HERE, "csrc", "list.cpp"), os.path.join(HERE, "csrc", "list.hip"),
           os.path.join(HERE, "csrc", "fp8.hip"), os.path.join(HERE, "csrc", "gemm.hip"),
           os.path.join(HERE, "csrc", "norm.hip"), os.path.join(HERE, "csrc", "vmm.cpp")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # IEEE fp32 step: no contraction into FMA, correctly rounded sqrt and
    # division, denormals kept.
    "-ffp-contract=off",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    # no packed-fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-I", os.path.join(HERE, "csrc"),
]


def _run(cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc failed building libdopt.so")


def build(verbose: bool = False) -> str:
    """Every source compiled anew, side by side, then linked in the library's place."""
    tmp = SO + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(int(os.environ.get("MAX_JOBS") or os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: _run([HIPCC, *FLAGS, "-c", so[0], "-o", so[1]], verbose), zip(SOURCES, objects)))
        _run([HIPCC, FLAGS[0], "-shared", *objects, "-o", tmp], verbose)
    os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    print(build(verbose=True))
