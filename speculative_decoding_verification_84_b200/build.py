"""Build the CUDA C-ABI library in-tree with nvcc for sm_100a.

    python -m speculative_decoding_verification_84_b200.build

produces ``speculative_decoding_verification_84_b200/lib/libspecverify.so``
from ``csrc/spec_verify.cu``, ``csrc/spec_draft.cu`` and the public header
``include/spec_verify.h``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", f) for f in ("spec_verify.cu", "spec_draft.cu")]
DEPS = [os.path.join(HERE, "csrc", f)
        for f in ("sv_common.cuh", "sv_host.cuh", "sv_generic.cuh", "sv_pass.cuh", "sv_small.cuh", "sv_topf.cuh",
                  "sv_bandit.cuh", "sv_tree.cuh", "sv_tc.cuh", "sv_lowrank.cuh", "sv_q8.cuh", "sv_beam.cuh")]
HEADER = os.path.join(ROOT, "include", "spec_verify.h")
LIB_DIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIB_DIR, "libspecverify.so")

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    newest = max(os.path.getmtime(f) for f in [*SRCS, HEADER, *DEPS])
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    objs = [f"{tmp}.{os.path.basename(src)}.o" for src in SRCS]
    flags = [*NVCC_FLAGS, *(["-Xptxas=-v"] if verbose else []), "-I", os.path.join(ROOT, "include")]
    try:
        # one compiler per source, side by side
        procs = [subprocess.Popen([nvcc(), *flags, "-c", src, "-o", obj]) for src, obj in zip(SRCS, objs)]
        codes = [p.wait() for p in procs]
        if any(codes):
            raise RuntimeError(f"nvcc failed on {[s for s, c in zip(SRCS, codes) if c]}")
        subprocess.check_call([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    finally:
        for f in (*objs, tmp):
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
