"""Build libjscan.so in place with hipcc for gfx950.

    python -m mamba_selective_scan_03_amd.build
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
# the library's sources: the selective scan and its producer, the gated recurrence, the int8 projection
SRCS = [os.path.join(HERE, "csrc", f) for f in ("jscan.hip", "gated_scan.hip", "int8_linear.hip")]
LIB = os.path.join(HERE, "libjscan.so")
# the microbenchmarks of the chip's ALU, matrix-core, LDS and HBM rates (measurement only)
MICRO_SRC = os.path.join(HERE, "csrc", "micro.hip")
MICRO_LIB = os.path.join(HERE, "libjscan_micro.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-ffp-contract=off",          # every fused multiply-add in the kernels is written out
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fPIC",
    "-Wall",
]


def _hipcc(args: list[str], verbose: bool):
    res = subprocess.run([HIPCC, *FLAGS, *args], capture_output=True, text=True)
    # hipcc's host pass does not know the device-only target feature; that note is harmless
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if ln.strip() and noise not in ln]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), file=sys.stderr)


def _compile(srcs: list[str], lib: str, verbose: bool) -> str:
    """Every source to an object of its own, side by side, then one shared library."""
    with tempfile.TemporaryDirectory(prefix="jscan_build_") as tmp, cf.ThreadPoolExecutor() as pool:
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in srcs]
        list(pool.map(lambda so: _hipcc(["-c", "-o", so[1], so[0]], verbose), zip(srcs, objs)))
        _hipcc(["-shared", "-o", lib + ".tmp", *objs], verbose)
    os.replace(lib + ".tmp", lib)
    return lib


def build(verbose: bool = False) -> str:
    """Compile the library and the microbenchmark library (always recompiles); returns the
    library's path."""
    with cf.ThreadPoolExecutor() as pool:
        micro = pool.submit(_compile, [MICRO_SRC], MICRO_LIB, verbose)
        lib = _compile(SRCS, LIB, verbose)
        micro.result()
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
