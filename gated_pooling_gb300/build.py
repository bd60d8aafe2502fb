"""Builds the CUDA library ``lib/libcsa_compressor.so`` in-tree with nvcc for sm_103a, and, where there is
g++ and this Python has its headers, the module ``lib/_csa_call`` through which the package calls it sooner than
through ctypes. The library needs nvcc alone and serves any Python; the module is this Python's.

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


def can_build_call() -> bool:
    """Whether the module can be built for this Python."""
    return shutil.which("g++") is not None and os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def _newer(out: str, inputs: List[str]) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in inputs)


def library_up_to_date() -> bool:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != CALL_SOURCE]
    return _newer(LIB, files + [os.path.join(INCLUDE, "csa_compressor.h"), os.path.abspath(__file__)])


def call_up_to_date() -> bool:
    return _newer(CALL, [os.path.join(CSRC, CALL_SOURCE), os.path.join(INCLUDE, "csa_compressor.h"), os.path.abspath(__file__)])


def up_to_date() -> bool:
    return library_up_to_date() and (call_up_to_date() or not can_build_call())


def _run(cmd: List[str], what: str) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what}:\n{res.stdout}{res.stderr}")
    return res.stdout + res.stderr


def _build_library(verbose: bool) -> None:
    cc = nvcc()

    def compile_one(src: str):
        obj = os.path.join(LIBDIR, os.path.splitext(src)[0] + ".o")
        return obj, f"=== {src}\n" + _run([cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc failed on {src}")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    log = "\n".join(text for _, text in results)
    with open(os.path.join(LIBDIR, "ptxas.log"), "w") as fh:
        fh.write(log)
    _run([cc, *ARCH, "-shared", "-o", LIB + ".tmp", *[obj for obj, _ in results]], "link failed")
    os.replace(LIB + ".tmp", LIB)
    if verbose:
        print(log)


def _build_call() -> None:
    _run([shutil.which("g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
          os.path.join(CSRC, CALL_SOURCE), "-o", CALL + ".tmp", "-L", LIBDIR, "-l:" + os.path.basename(LIB),
          "-Wl,-rpath,$ORIGIN"], f"g++ failed on {CALL_SOURCE}")
    os.replace(CALL + ".tmp", CALL)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is missing or stale; the module is left out where it cannot be built."""
    os.makedirs(LIBDIR, exist_ok=True)
    if force or not library_up_to_date():
        _build_library(verbose)
    if can_build_call() and (force or not call_up_to_date()):
        _build_call()
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
