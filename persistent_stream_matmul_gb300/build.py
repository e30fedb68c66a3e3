"""Build the sm_103a GEMM library in-tree: ``libpsm_gemm.so`` beside this file."""
from __future__ import annotations

import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpsm_gemm.so")
# each translation unit and the headers it includes
UNITS = {
    "gemm.cu": ("gemm_kernel.cuh", "upload.cuh", "ptx.cuh", "sched.cuh", "gemm.h"),
    "moe.cu": ("ptx.cuh", "rows.cuh", "host.cuh", "upload.cuh", "gemm.h", "gemm_moe.h"),
    "grouped.cu": ("grouped_kernel.cuh", "grouped_sched.cuh", "join.cuh", "host.cuh", "upload.cuh", "ptx.cuh", "gemm.h", "gemm_moe.h"),
    "scaled_rows.cu": ("ptx.cuh", "rows.cuh", "host.cuh", "upload.cuh", "gemm.h", "gemm_scaled.h"),
    "packed.cu": ("gemm.h", "gemm_scaled.h"),
    "scaled.cu": ("scaled_few.cuh", "scaled_kernel.cuh", "rows.cuh", "join.cuh", "host.cuh", "upload.cuh", "ptx.cuh", "gemm.h", "gemm_scaled.h"),
}
SOURCES = [os.path.join(CSRC, f) for f in UNITS]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _header(name: str) -> str:
    return os.path.join(CSRC if name.endswith(".cuh") else INCLUDE, name)


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in inputs)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is missing or older than its sources, the units in
    parallel, and link the library."""
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    suffix = ".tmp%d" % os.getpid()
    objects, jobs = [], []
    for source, headers in UNITS.items():
        src = os.path.join(CSRC, source)
        obj = src[:-3] + ".o"
        objects.append(obj)
        if force or _stale(obj, [src, *map(_header, headers)]):
            cmd = [nvcc(), *flags, "-c", "-o", obj + suffix, src]
            jobs.append((subprocess.Popen(cmd), cmd, obj))
    failed = [cmd for job, cmd, _ in jobs if job.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, obj in jobs:
        os.replace(obj + suffix, obj)
    if jobs or _stale(LIB, objects):
        subprocess.check_call([nvcc(), *ARCH, "-shared", "-o", LIB + suffix, *objects])
        os.replace(LIB + suffix, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
