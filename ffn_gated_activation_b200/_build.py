"""Build of the native library libsitu_glu.so (nvcc, sm_100a, in-tree).

nvcc cross-compiles for sm_100a without a GPU, so this runs anywhere the CUDA
toolkit is installed.  The shared object is written next to this file so that
it travels with the source tree.
"""
from __future__ import annotations

import concurrent.futures
import hashlib
import os
import shutil
import subprocess

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SOURCES = [os.path.join(PKG_DIR, "csrc", n) for n in ("situ_glu.cu", "situ_norm.cu", "situ_moe.cu", "situ_nvfp4.cu")]
HEADERS = [os.path.join(ROOT, "include", "situ_glu.h")] + [
    os.path.join(PKG_DIR, "csrc", n) for n in ("situ_device.cuh", "situ_host.cuh", "situ_fused_gemm.cuh")]
LIBRARY = os.path.join(PKG_DIR, "libsitu_glu.so")
OBJECT_DIR = os.path.join(PKG_DIR, "build")  # one object per source, kept for the next build

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def is_stale(output: str = LIBRARY) -> bool:
    if not os.path.exists(output):
        return True
    t = os.path.getmtime(output)
    return any(os.path.getmtime(p) > t for p in SOURCES + HEADERS)


def _compile(source: str, force: bool, extra_flags) -> str:
    """The object file of one source, compiled unless it is up to date."""
    flags = [*NVCC_FLAGS, *extra_flags]
    tag = hashlib.sha256(" ".join(flags).encode()).hexdigest()[:8]  # other flags, another object
    obj = os.path.join(OBJECT_DIR, f"{os.path.splitext(os.path.basename(source))[0]}.{tag}.o")
    if not force and os.path.exists(obj):
        t = os.path.getmtime(obj)
        if all(os.path.getmtime(p) <= t for p in [source] + HEADERS):
            return obj
    tmp = f"{obj}.tmp{os.getpid()}.o"
    subprocess.run([nvcc(), *flags, "-c", "-I", os.path.join(ROOT, "include"), source, "-o", tmp], check=True)
    os.replace(tmp, obj)
    return obj


def build_library(force: bool = False, output: str = LIBRARY, extra_flags=()) -> str:
    """Compile the CUDA sources (one nvcc per source, side by side) and link
    them into ``output`` unless it is up to date."""
    if not force and not is_stale(output):
        return output
    os.makedirs(OBJECT_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = list(pool.map(lambda s: _compile(s, force, extra_flags), SOURCES))
    tmp = output + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), *NVCC_FLAGS, *extra_flags, "-shared", *objects, "-o", tmp], check=True)
    os.replace(tmp, output)
    return output


if __name__ == "__main__":
    print(build_library(force=True))
