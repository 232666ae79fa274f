"""Builds libdspark.so for gfx950 in-tree with hipcc.

    python -m vocab_wide_draft_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", *at) for at in
           (("dspark.hip",), ("logits", "logits.hip"), ("head", "head.hip"), ("beam", "beam.hip"))]
OUT = os.path.join(HERE, "libdspark.so")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off",                      # every fused multiply-add is written explicitly
    "-fno-gpu-flush-denormals-to-zero",       # binary32 subnormal weights are kept
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"),
]


def build(verbose: bool = False) -> str:
    """Compiles the sources side by side and links them."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    with tempfile.TemporaryDirectory() as work:
        objects = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        cmds = [[hipcc, *FLAGS, "-c", "-o", o, s] for s, o in zip(SOURCES, objects)]
        running = []
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append(subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True))
        errors = [p.communicate()[1] for p in running]
        for p, err in zip(running, errors):
            if p.returncode != 0:
                err = "\n".join(l for l in err.splitlines() if "packed-fp32-ops" not in l)
                raise RuntimeError(f"hipcc failed ({p.returncode}):\n{err}")
        tmp = OUT + ".tmp"
        cmd = [hipcc, "--offload-arch=gfx950", "-shared", "-o", tmp, *objects]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stderr}")
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
