"""Build libaq.so (the C-ABI library) in-tree with hipcc for gfx950.

    python -m group_wise_affine_aq_amd.build        # compile everything

Each source compiles to an object in ``_build/`` in parallel, then one shared
library is linked next to this file.  Packed-fp32 instruction selection is
switched off for all device code.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libaq.so")
ARCH = os.environ.get("AQ_OFFLOAD_ARCH", "gfx950")

SOURCES = ["aq_api.cpp", "aq_quant.hip", "aq_qmv.hip", "aq_qmvm.hip", "aq_qmm.hip", "aq_fp.hip",
           "aq_kv.hip", "aq_attn.hip", "aq_attn_masked.hip", "aq_weigh.hip", "aq_rope.hip", "aq_evict.hip",
           "aq_prompt.hip", "aq_bench.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]
# Matrix products of the prompt kernels have their sums in ordinary registers: with heads of 256 the
# compiler puts them into accumulation registers and moves all 128 out and back around each branch that
# may rescale them (8192 tokens of 32 heads of 256: 1520 us so, 1165 us with this).
MORE_FLAGS = {"aq_prompt.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, *MORE_FLAGS.get(src, []), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stderr}")
    # the host pass warns that it does not know the packed-fp32 feature: harmless
    noise = "packed-fp32-ops' is not a recognized feature"
    msgs = [l for l in res.stderr.splitlines() if l.strip() and noise not in l]
    if msgs:
        sys.stderr.write("\n".join(msgs) + "\n")
    return obj


def build(jobs: int | None = None) -> str:
    """Compile every source and link libaq.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), os.cpu_count() or 1, 8)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
