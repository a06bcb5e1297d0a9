"""Compile the HIP library ``libgdn_tree.so`` for gfx950 with hipcc.

Usage: ``python -m gated_deltanet_tree_gdn_amd.build`` (or
``__graft_entry__.build()``).  The library is built in-tree, next to this
file, so it travels with the source tree.
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
LIB = os.path.join(PKG, "libgdn_tree.so")

SOURCES = ["gdn_tree_api.cpp", "gdn_simple.hip", "gdn_fast.hip", "gdn_verify_ws.hip", "gdn_commit_verify.hip", "gdn_commit.hip", "gdn_draft.hip", "gdn_branch.hip", "gdn_static.hip", "gdn_split.hip",
           "gdn_layer_api.cpp", "gdn_norm.hip", "gdn_decode.hip", "gdn_prefill.hip", "gdn_linear.hip"]

# Packed fp32 VALU ops are switched off for all device code.
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the library)")


def build(verbose: bool = False, extra_flags=()) -> str:
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *HIP_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-o", tmp, *srcs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass reports the device-only feature flag as unknown
    noise = "'-packed-fp32-ops' is not a recognized feature"
    errs = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{errs}")
    if verbose and errs.strip():
        print(errs, file=sys.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
