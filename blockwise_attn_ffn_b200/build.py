"""Builds libbpt.so in-tree with nvcc for sm_100a.

    python -m blockwise_attn_ffn_b200.build

The library is two translation units (csrc/bpt_api.cu, the layer calls, and
csrc/ops_api.cu, the attention operators and the key-value cache, each
including its kernel headers), compiled side by side and linked against the
static CUDA runtime; the driver API entry point they need (tensor-map
encoding) is resolved at run time, so no libcuda stub is linked.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libbpt.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]
UNITS = ["bpt_api.cu", "ops_api.cu"]


def sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
            if f.endswith((".cu", ".cuh"))] + [os.path.join(INCLUDE, "bpt.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def nvcc() -> str:
    for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: libbpt.so cannot be built")


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile the units of csrc/ into libbpt.so (skipped when up to date)."""
    if not force and up_to_date():
        return LIB
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as obj_dir:
        objs, jobs = [], []
        for unit in UNITS:
            objs.append(os.path.join(obj_dir, unit + ".o"))
            cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I" + INCLUDE, "-I" + CSRC, "-c",
                   os.path.join(CSRC, unit), "-o", objs[-1]]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                         text=True))
        outs = [j.communicate()[0] for j in jobs]
        for job, out in zip(jobs, outs):
            if job.returncode != 0:
                raise RuntimeError("nvcc failed:\n" + out)
            if verbose and out:
                print(out)
        r = subprocess.run([nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
                            "-Xcompiler", "-fPIC", *objs, "-o", tmp], capture_output=True,
                           text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
