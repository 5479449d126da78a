"""Build libecho.so (gfx950) from csrc/ with hipcc, in-tree.

Flags: -ffp-contract=off keeps every a*b+c as two rounded operations (the
results must match the CPU definition bit for bit); packed fp32 instructions
are disabled; fp32 denormals are kept (no flush to zero).
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libecho.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def sources():
    return [os.path.join(CSRC, f) for f in ("echo_api.hip", "echo_block_api.hip", "echo_int4_api.hip", "echo_cache_api.hip")]


# test-only device code: the kernels' helpers evaluated on their own, built
# with the library's flags (loaded by tests/test_gpu_*.py only)
CHECK_SRC = os.path.join(ROOT, "tests", "c", "recip_scale_check.hip")
CHECK_LIB = os.path.join(ROOT, "tests", "c", "librecip_scale_check.so")


def _hipcc(args, what: str, verbose: bool) -> None:
    cmd = [HIPCC, *HIP_FLAGS, *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 target feature and says so; drop that line
    msgs = [l for l in (r.stderr or "").splitlines() if "is not a recognized feature for this target" not in l]
    if r.returncode != 0:
        sys.stderr.write("\n".join(msgs) + "\n")
        raise RuntimeError(f"hipcc failed ({r.returncode}) building {what}")
    if msgs and verbose:
        sys.stderr.write("\n".join(msgs) + "\n")


def build(verbose: bool = False) -> str:
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in sources()]
        inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
        with ThreadPoolExecutor(max_workers=len(objs) + 1) as pool:
            jobs = [pool.submit(_hipcc, [*inc, "-c", s, "-o", o], s, verbose) for s, o in zip(sources(), objs)]
            jobs.append(pool.submit(build_check, verbose))
            for j in jobs:
                j.result()
        _hipcc(["-shared", *objs, "-o", LIB + ".tmp"], LIB, verbose)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def build_check(verbose: bool = False) -> str:
    _hipcc(["-shared", "-I", os.path.join(ROOT, "include"), "-I", CSRC, CHECK_SRC, "-o", CHECK_LIB + ".tmp"], CHECK_LIB, verbose)
    os.replace(CHECK_LIB + ".tmp", CHECK_LIB)
    return CHECK_LIB


if __name__ == "__main__":
    print(build(verbose=True))
