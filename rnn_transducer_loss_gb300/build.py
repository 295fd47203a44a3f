"""Build librnnt_gb300.so in-tree with nvcc for sm_103a (no CMake; one translation unit for
the loss and one for each pair of operators around it, compiled side by side)."""
from __future__ import annotations

import os
import subprocess
import sys
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SRCS = [os.path.join(CSRC, f) for f in ("rnnt_gb300.cu", "rnnt_embed.cu", "rnnt_beam.cu",
                                            "rnnt_distill.cu", "rnnt_sample.cu")]
DEPS = [os.path.join(CSRC, f) for f in ("rnnt_labels.cuh", "rnnt_rows.cuh")]
HDR = os.path.join(ROOT, "include", "rnnt_gb300.h")
LIB = os.path.join(PKG, "librnnt_gb300.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-Xcompiler", "-fPIC,-O2",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in (*SRCS, *DEPS, HDR, __file__))


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [nvcc(), *NVCC_FLAGS, *(extra or []), "-I", os.path.join(ROOT, "include")]
    t0 = time.time()
    objs = [f"{tmp}.{i}.o" for i in range(len(SRCS))]
    try:
        jobs = [subprocess.Popen([*flags, "-c", src, "-o", obj], stdout=subprocess.PIPE,
                                 stderr=subprocess.STDOUT, text=True)
                for src, obj in zip(SRCS, objs)]
        logs = [j.communicate()[0] for j in jobs]
        failed = any(j.returncode for j in jobs)
        if not failed:
            res = subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", *objs, "-o", tmp],
                                 stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            logs.append(res.stdout)
            failed = res.returncode != 0
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    if failed or verbose:
        sys.stderr.write("".join(logs))
    if failed:
        raise RuntimeError("nvcc failed building librnnt_gb300.so")
    if verbose:
        sys.stderr.write(f"built {LIB} in {time.time() - t0:.1f}s\n")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
