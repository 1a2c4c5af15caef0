"""Build libzero.so (sm_103a) in-tree with nvcc; translation units compile in parallel."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libzero.so")
OBJ_DIR = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]
SOURCES = ["zero_plan.cpp", "zero_step.cu", "zero_offload.cpp", "zero_adamw.cu",
           "zero_linear.cu", "zero_norm.cu", "zero_gated.cu", "zero_muon.cu"]
# the host AdamW must round every fp32 operation separately, like the GPU kernel; without errno
# bookkeeping its square root (an exact IEEE operation either way) lets the loop vectorise, and
# without trapping math the compiler may evaluate the fp16 rounding's one fp32 addition for
# every element (results are the same IEEE values; no floating-point exception flag is read),
# which keeps that loop free of branches and vectorised too
EXTRA = {"zero_offload.cpp": ["-Xcompiler", "-ffp-contract=off", "-Xcompiler", "-fno-fast-math",
                              "-Xcompiler", "-fno-math-errno", "-Xcompiler", "-fno-trapping-math"]}


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    procs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ_DIR, src + ".o")
        objs.append(obj)
        cmd = [NVCC, *GENCODE, *FLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((cmd, subprocess.Popen(cmd)))
    for cmd, pr in procs:
        if pr.wait() != 0:
            raise RuntimeError("compile failed: " + " ".join(cmd))
    tmp = f"{LIB}.{os.getpid()}.tmp"             # renamed into place: never half-written
    subprocess.run([NVCC, *GENCODE, "-shared", *objs, "-o", tmp, "-lpthread"], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
