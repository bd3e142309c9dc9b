"""Build ``libconvrot.so`` in-tree with hipcc for gfx950.

Usage: ``python -m w8a8_rotated_int8_convrot_amd.build`` (or ``build()``).
The library is placed next to this file, where ``binding`` looks for it.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libconvrot.so")
SOURCES = ("convrot_api.hip", "rotate_quant.hip", "gemm_i8.hip", "gemm_grouped.hip", "gemm_lora.hip", "lora.hip",
           "default_path.hip", "block_norm.hip", "operators_api.hip", "mfma_probe.hip")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # every float operation is one IEEE operation in the written order: the
    # rotation must reproduce the same sums bit for bit, and fused multiply-adds
    # are written out explicitly where wanted
    "-ffp-contract=off",
    # fp32 '/' is the correctly rounded IEEE division
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # keep small per-thread arrays (staging pointers) in registers instead of
    # letting the compiler move them into LDS, which the GEMM tiles fill
    "-mllvm", "-disable-promote-alloca-to-lds",
    "-Wall",
]
LINK_FLAGS = ["--offload-arch=gfx950", "-fPIC", "-shared"]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp%d" % os.getpid()

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        # the host pass warns that it does not know the packed-fp32 feature
        noise = "is not a recognized feature for this target"
        msgs = [l for l in (res.stdout + res.stderr).splitlines() if noise not in l]
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
        if verbose and msgs:
            print("\n".join(msgs), flush=True)

    # the sources side by side, then one link
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, s.replace(".hip", ".o")) for s in SOURCES]
        cmds = [[HIPCC, *FLAGS, "-c", "-o", o, os.path.join(CSRC, s)] for s, o in zip(SOURCES, objs)]
        with concurrent.futures.ThreadPoolExecutor(min(len(SOURCES), 8)) as pool:
            list(pool.map(run, cmds))
        run([HIPCC, *LINK_FLAGS, "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
