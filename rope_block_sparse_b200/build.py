"""Build libh3a.so in-tree for sm_100a with nvcc, and where torch is installed its
binding (csrc/binding.cpp) with g++.

    python -m rope_block_sparse_b200.build [--force] [--verbose]
    python rope_block_sparse_b200/build.py         # the library alone needs no torch

Each .cu file is compiled to an object under ``_build/`` (in parallel), then
linked into ``rope_block_sparse_b200/libh3a.so`` with the CUDA runtime linked
statically, so the library loads on a machine without a GPU driver (calls
that reach CUDA then fail with H3A_ERR_CUDA).  ``ptxas -v`` output (registers,
spills, shared memory) is kept in ``_build/<name>.ptxas.txt``.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libh3a.so")
SOURCES = ["h3a_api.cu", "prologue.cu", "router.cu", "attention.cu", "selftest.cu", "route_noalloc.cu", "dit_ops.cu",
           "rope.cu", "rmsnorm.cu", "packed_plan.cu", "packed_tiles.cu", "packed_rows.cu", "packed_combine.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libh3a")


def _newer(files: list, than: str) -> bool:
    if not os.path.exists(than):
        return True
    t = os.path.getmtime(than)
    return any(os.path.getmtime(f) > t for f in files)


def _library_inputs() -> list:
    return [os.path.join(INCLUDE, "h3a.h")] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp"]


def _binding_inputs() -> list:
    return [os.path.join(INCLUDE, "h3a.h"), os.path.join(CSRC, "binding.cpp")]


def _torch():
    """The installed torch, or None if there is none with CUDA (one that is broken raises)."""
    try:
        import torch
    except ModuleNotFoundError as e:
        if e.name != "torch":
            raise
        return None
    return torch if torch.version.cuda else None


def binding_path(torch) -> str:
    """The binding for this torch and Python.  It uses torch's C++ classes and Python's API as they were when it
    was compiled, so its name says which, as an extension module's does, and no other is loaded or kept."""
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(PKG, f"_binding.torch-{torch.__version__}.abi{abi}.{sys.implementation.cache_tag}.so")


def needs_build() -> bool:
    torch = _torch()
    return _newer(_library_inputs(), LIB) or (torch is not None and _newer(_binding_inputs(), binding_path(torch)))


def _binding_cmd(torch, out: str) -> list:
    """g++ of the torch binding; it finds libh3a.so beside itself."""
    import sysconfig

    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    includes = [os.path.join(root, "include"), sysconfig.get_paths()["include"], cuda]
    libs = os.path.join(root, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, *[x for i in includes for x in ("-isystem", i)], os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L", libs, "-L", PKG, "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}", "-l:libh3a.so", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_cuda", "-ltorch_python"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is not up to date; without torch the library alone, whose C ABI does not need it."""
    if force or _newer(_library_inputs(), LIB):
        _build_library(verbose)
    torch = _torch()
    if torch is None:
        print("no torch with CUDA: libh3a.so is built, its torch binding is not", file=sys.stderr)
    elif force or _newer(_binding_inputs(), binding_path(torch)):
        tmp = binding_path(torch) + f".tmp{os.getpid()}"
        subprocess.check_call(_binding_cmd(torch, tmp))
        os.replace(tmp, binding_path(torch))
    return LIB


def _build_library(verbose: bool) -> None:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        log = open(os.path.join(BUILD, src.replace(".cu", ".ptxas.txt")), "w")
        procs.append((src, obj, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT), log))
    failed = []
    for src, obj, p, log in procs:
        p.wait()
        log.close()
        if p.returncode != 0:
            failed.append(src)
        if verbose or p.returncode != 0:
            sys.stderr.write(open(log.name).read())
    if failed:
        raise RuntimeError(f"nvcc failed on {failed}")
    tmp = LIB + f".tmp{os.getpid()}"
    link = [nvcc, *ARCH, "-shared", "-o", tmp, "-Xlinker", "-soname=libh3a.so", *[o for _, o, _, _ in procs], "-cudart", "static"]
    subprocess.check_call(link)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
