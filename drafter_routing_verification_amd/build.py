"""Compiles libwhiflash.so for gfx950 in-tree with hipcc.

    python -m drafter_routing_verification_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libwhiflash.so")
SOURCES = ["api.hip", "sweep.hip", "finalize.hip", "router.hip", "entropy.hip", "catchup.hip", "round.hip", "early_exit.hip",
           "noalloc.hip", "api_rounds.hip", "rules.hip", "history.hip", "attend.hip", "pages.hip",
           "api_decode.hip", "rotary.hip", "cache8.hip", "attend8.hip", "logprobs.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libwhiflash)")


def command(out: str) -> list[str]:
    return [
        hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
        "-Wall", "-Wno-unused-command-line-argument",
        # no packed fp32 VALU instructions (v_pk_add/mul/fma_f32): the compiler would
        # otherwise pair the kernels' scalar float32 operations into them; all float
        # arithmetic here is meant to run as scalar float32 VALU instructions
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, "-I", CSRC, "-o", out,
    ] + [os.path.join(CSRC, s) for s in SOURCES]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    cmd = command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed with exit code {res.returncode}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
