"""Build libmoe_mxfp4.so in-tree with hipcc for gfx950.

    python -m mxfp4_weight_expert_amd.build

Always recompiles, a few sources at a time. Packed-FP32 VALU ops are disabled for device code.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe_mxfp4.so")
SOURCES = ["api.hip", "route.hip", "sort.hip", "quant.hip", "gemm.hip", "gemm_tiled.hip",
           "finalize.hip", "pack.hip", "dispatch.hip", "combine.hip", "w4_bf16.hip", "w4_fp16.hip", "ops_api.hip"]
ARCH = "gfx950"
JOBS = 6  # sources compiled at once


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def build(verbose: bool = False) -> str:
    cc = hipcc()
    flags = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-I",
             os.path.join(ROOT, "include"),
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        proc = subprocess.run(cmd, capture_output=True, text=True)
        if proc.returncode != 0:
            sys.stderr.write(proc.stdout + proc.stderr)
            raise RuntimeError(f"hipcc failed with status {proc.returncode}")

    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objs:
        pairs = [(os.path.join(CSRC, s), os.path.join(objs, s + ".o")) for s in SOURCES]
        with ThreadPoolExecutor(JOBS) as pool:
            list(pool.map(lambda p: run([cc, *flags, "-c", p[0], "-o", p[1]]), pairs))
        run([cc, f"--offload-arch={ARCH}", "-shared", *[o for _, o in pairs], "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
