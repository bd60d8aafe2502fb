"""Builds the CUDA library ``lib/libcsa_compressor.so`` in-tree with nvcc for sm_103a, and the Python
module ``lib/_csa_call`` through which the package calls it.

Each translation unit compiles in its own nvcc process, in parallel, then one link.
ptxas resource usage (registers, spills, shared memory) is kept in ``lib/ptxas.log``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
from typing import List

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libcsa_compressor.so")
CALL = os.path.join(LIBDIR, "_csa_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
CALL_SOURCE = "csa_call.cpp"
SOURCES = ["csa_fwd.cu", "csa_bwd.cu", "csa_api.cu", "csa_noalloc.cu", "csa_kpool.cu",
           "csa_rope.cu", "csa_cache.cu", "csa_append.cu", "csa_step.cu", "csa_attn.cu",
           "csa_attn_prefix.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def cxx() -> str:
    path = shutil.which("g++")
    if path is None:
        raise RuntimeError("g++ not found: it is required to build the package's calls")
    return path


def _inputs() -> List[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    return files + [os.path.join(INCLUDE, "csa_compressor.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALL))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str):
        obj = os.path.join(LIBDIR, os.path.splitext(src)[0] + ".o")
        if src == CALL_SOURCE:
            cmd = [cxx(), "-O2", "-std=c++17", "-fPIC", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE]
        else:
            cmd = [cc, *ARCH, *FLAGS]
        cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, res

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        results = list(ex.map(compile_one, [*SOURCES, CALL_SOURCE]))
    log = []
    for src, _, res in results:
        log.append(f"=== {src}\n{res.stdout}{res.stderr}")
        if res.returncode != 0:
            raise RuntimeError(f"the compiler failed on {src}:\n{res.stdout}{res.stderr}")
    with open(os.path.join(LIBDIR, "ptxas.log"), "w") as fh:
        fh.write("\n".join(log))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for src, o, _ in results if src != CALL_SOURCE]]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}{res.stderr}")
    os.replace(tmp, LIB)
    tmp = CALL + ".tmp"
    cmd = [cxx(), "-shared", "-o", tmp, results[-1][1], "-L", LIBDIR, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}{res.stderr}")
    os.replace(tmp, CALL)
    if verbose:
        print("\n".join(log))
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
