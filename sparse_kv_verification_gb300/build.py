"""Builds the CUDA library libdustin.so in-tree (sm_103a, one -gencode).

Each translation unit is compiled by nvcc in parallel, then linked into a
shared library with the static CUDA runtime.  The result lives in
``sparse_kv_verification_gb300/_build/`` and is rebuilt only when a source or
header is newer.  Usage: ``python -m sparse_kv_verification_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
from typing import List

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libdustin.so")

SOURCES = ["api.cu", "score.cu", "select.cu", "attn_sparse.cu", "attn_dense.cu",
           "attn_ml.cu", "quest.cu", "tokens.cu", "kv_pages.cu",
           "attn_prefix.cu", "kv4_cache.cu", "attn_kv4.cu", "attn_kv4_d64.cu",
           "attn_kv4_d128.cu", "logprobs.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required")
    return path


def _inputs() -> List[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "dustin.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False,
          extra: List[str] | None = None, out: str | None = None) -> str:
    """Compiles the library if needed and returns its path.  `extra` adds
    nvcc flags (e.g. -D tunables); `out` builds to another path (always
    rebuilt)."""
    if out is None and not force and up_to_date():
        return LIB
    lib_path = out or LIB
    obj_dir = os.path.join(os.path.dirname(os.path.abspath(lib_path)),
                           "obj_" + os.path.basename(lib_path)) if out else BUILD
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src),
               "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib_path + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(force="--force" in sys.argv, verbose=v,
                extra=["-Xptxas", "-v"] if v else None))
