"""Build libmxmoe.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled in parallel, then linked into
``mxfp8_block_scaled_moe_gb300/libmxmoe.so`` with a static CUDA runtime, so
the library needs nothing but the NVIDIA driver at run time.  Beside it, g++
compiles ``csrc/binding.cpp`` against the installed PyTorch's headers into the
native half of ``block_ops``, ``_binding.so``.  Object files go to ``_build/`` at
the repository root.  No CMake.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libmxmoe.so")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")

SOURCES = ["api.cu", "quant.cu", "route.cu", "finalize.cu", "gemm.cu", "gemm2sm.cu", "noalloc.cu",
           "router.cu", "norm.cu", "linear.cu", "linear_pair.cu", "balance.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmxmoe.so")


def _binding_command(out: str) -> list:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            "-I" + INCLUDE, "-I" + os.path.join(torch, "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
            "-o", out, os.path.join(CSRC, "binding.cpp"), "-L" + os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + \
        [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libmxmoe.so."""
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= _deps_mtime()
                         for p in (LIB_PATH, BINDING_PATH)):
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        log = open(os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".log"), "w")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((src, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT), log))
        objs.append(obj)
    log = open(os.path.join(BUILD_DIR, "binding.log"), "w")
    binding_tmp = BINDING_PATH + ".tmp"
    procs.append(("binding.cpp", subprocess.Popen(_binding_command(binding_tmp), stdout=log,
                                                 stderr=subprocess.STDOUT), log))
    failed = []
    for src, p, log in procs:
        rc = p.wait()
        log.close()
        if rc != 0:
            failed.append(src)
    if failed:
        msgs = []
        for src in failed:
            with open(os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".log")) as f:
                msgs.append(f"--- {src}\n" + f.read()[-4000:])
        raise RuntimeError("compilation failed:\n" + "\n".join(msgs))
    tmp = LIB_PATH + ".tmp"
    link = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB_PATH)
    os.replace(binding_tmp, BINDING_PATH)
    if verbose:
        for src in SOURCES:
            with open(os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".log")) as f:
                sys.stdout.write(f.read())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
