"""Build libmoe_fp4.so (gfx950) in-tree with hipcc.

    python -m block_scaled_fp4_gather_amd.build

Packed-fp32 VALU forms are disabled for all device code
(-target-feature -packed-fp32-ops); the host pass warns that it does not
know the feature, which is harmless.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe_fp4.so")
SOURCES = ["api.hip", "prepare.hip", "decode_path.hip", "prefill.hip", "prefill_a8.hip", "mxfp8.hip",
           "router.hip", "fp8_linear.hip", "block_norm.hip", "block_api.hip",
           "fp4_quant.hip", "fp4_linear.hip", "grouped.hip", "routes.hip", "experts_api.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"


FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-command-line-argument"]


def _run(cmd: list[str], made: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed building {made}")


def build(verbose: bool = False) -> str:
    """Compiles the sources side by side, up to 8 (or MAX_JOBS) at a time, and links them."""
    tmp = LIB + ".tmp"
    jobs = max(1, min(8, int(os.environ.get("MAX_JOBS") or os.cpu_count() or 1)))
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        with concurrent.futures.ThreadPoolExecutor(jobs) as pool:
            list(pool.map(lambda s, o: _run([HIPCC, *FLAGS, "-c", "-o", o, os.path.join(CSRC, s)], s, verbose),
                          SOURCES, objects))
        _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-o", tmp, *objects], os.path.basename(LIB), verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
