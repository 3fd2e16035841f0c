"""Builds the C-ABI library ``libfswin.so`` in-tree with nvcc for sm_100a."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libfswin.so")
SOURCES = ["api.cu", "fwd.cu", "bwd.cu", "small.cu", "block.cu", "noalloc.cu", "wide.cu", "lrbias.cu", "relbias.cu",
           "relbias_small.cu", "resnorm.cu", "resnorm_bwd.cu", "mlp.cu", "mlp_small.cu"]
HEADERS = ["dgeo.cuh", "geometry.cuh", "kernels.cuh", "mlp.cuh", "ptx.cuh", "relbias.cuh", "resnorm.cuh",
           "rows.cuh", "schedule.cuh", "tile_io.cuh"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "fswin.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source for sm_100a and link libfswin.so (no-op when fresh)."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = nvcc_path()
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
             "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags += ["-Xptxas", "-v"]
    objs = [os.path.join(BUILD, src.replace(".cu", ".o")) for src in SOURCES]

    def compile_one(src: str, obj: str) -> None:
        subprocess.check_call([nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj])

    with ThreadPoolExecutor(max_workers=max(1, min(len(SOURCES), os.cpu_count() or 1))) as pool:
        for done in [pool.submit(compile_one, src, obj) for src, obj in zip(SOURCES, objs)]:
            done.result()
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", tmp,
                           "-lcudart"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
