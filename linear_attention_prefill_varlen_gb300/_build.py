"""Builds the CUDA library in-tree with nvcc (sm_103a only)."""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SRC_DIR = os.path.join(PKG_DIR, "csrc")
OBJ_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libkdaconv.so")

# No fast-math: the taps are explicit fmaf calls, divisions and expf stay IEEE
# unless the source asks otherwise, and denormals are kept.
NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libkdaconv.so")


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(SRC_DIR, "*.cu")))


def _newest_header() -> float:
    headers = glob.glob(os.path.join(SRC_DIR, "*.cuh")) + glob.glob(
        os.path.join(ROOT, "include", "*.h"))
    return max(os.path.getmtime(p) for p in [*headers, __file__])


def build(force: bool = False, extra_flags: list[str] | None = None, out: str = LIB_PATH) -> str:
    """Compiles csrc/*.cu (in parallel, one object each) into libkdaconv.so next
    to this file.  An object newer than its source and every header is kept."""
    sources, headers = _sources(), _newest_header()
    newest = max(headers, *(os.path.getmtime(p) for p in sources))
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest and not extra_flags:
        return out
    nvcc = nvcc_path()
    os.makedirs(OBJ_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory(dir=OBJ_DIR) as work:
        def compile_one(src: str) -> str:
            name = os.path.basename(src)[:-3] + ".o"
            kept = os.path.join(OBJ_DIR, name)
            if not force and not extra_flags and os.path.exists(kept) and (
                    os.path.getmtime(kept) >= max(headers, os.path.getmtime(src))):
                return kept
            obj = os.path.join(work, name)
            subprocess.run([nvcc, *NVCC_FLAGS, *(extra_flags or []), "-I",
                            os.path.join(ROOT, "include"), "-c", "-o", obj, src], check=True)
            if extra_flags:
                return obj
            os.replace(obj, kept)
            return kept

        with ThreadPoolExecutor(max_workers=len(sources)) as pool:
            objects = list(pool.map(compile_one, sources))
        tmp = out + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *NVCC_FLAGS, "-shared", "-o", tmp, *objects], check=True)
        os.replace(tmp, out)
    return out
