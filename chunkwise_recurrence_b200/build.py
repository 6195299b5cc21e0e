"""Compiles libgdr (chunkwise_recurrence_b200/libgdr.so) for sm_100a with nvcc,
and the PyTorch marshalling of some of its entries (_binding.*.so) with g++.

Usage: python -m chunkwise_recurrence_b200.build [--force]
The library is built in-tree so that it travels with the source tree.  It needs
no PyTorch: where PyTorch (or a header, or g++) is missing, only the marshalling
is left out, and build() says so.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdr.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-cudart", "static",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libgdr cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def binding_path() -> str:
    """The extension for this Python and this PyTorch: another one's has
    another name, so that an extension is never loaded into a PyTorch that it
    was not compiled against."""
    import torch
    return os.path.join(PKG, f"_binding.{sysconfig.get_config_var('SOABI')}-"
                             f"torch{torch.__version__}.so")


def binding_needs() -> str | None:
    """What is missing to build the extension, or None."""
    try:
        import torch
    except ImportError:
        return "PyTorch"
    root = os.path.dirname(torch.__file__)
    for what, path in (
            ("PyTorch's headers",
             os.path.join(root, "include", "torch", "csrc", "autograd",
                          "python_variable.h")),
            ("a PyTorch with CUDA", os.path.join(root, "lib",
                                                 "libc10_cuda.so")),
            ("Python's headers",
             os.path.join(sysconfig.get_paths()["include"], "Python.h"))):
        if not os.path.exists(path):
            return what
    if not shutil.which("g++"):
        return "g++"
    try:
        _nvcc()                  # (CUDA's headers stand beside it)
    except RuntimeError:
        return "nvcc"
    return None


def _binding_stale() -> bool:
    path = binding_path()
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    deps = [BINDING_SRC, __file__] + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build_binding(force: bool = False) -> str:
    """The CPython extension that hands PyTorch tensors to libgdr."""
    missing = binding_needs()
    if missing:
        raise RuntimeError(f"{missing} not found: the binding cannot be built")
    if not force and not _binding_stale():
        return binding_path()
    import torch
    root = os.path.dirname(torch.__file__)
    path = binding_path()
    tmp = path + ".tmp"
    subprocess.run(
        [shutil.which("g++"), "-O2", "-std=c++17", "-fPIC",
         "-fvisibility=hidden", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
         "-I", os.path.join(root, "include"),
         "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())),
                            "include"),
         BINDING_SRC, "-o", tmp, "-L", PKG, "-l:libgdr.so",
         "-Wl,-rpath,$ORIGIN", "-L", os.path.join(root, "lib"), "-lc10",
         "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], check=True)
    os.replace(tmp, path)
    return path


def _build_binding_if_possible(force: bool = False) -> None:
    missing = binding_needs()
    if missing:
        print(f"{missing} not found: libgdr.so is built without its PyTorch "
              "binding", file=sys.stderr)
    else:
        build_binding(force)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        _build_binding_if_possible()
        return LIB
    nvcc = _nvcc()
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src,
               "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        return obj

    # (with -v one after another, so that what ptxas says stays together)
    jobs = 1 if verbose else os.cpu_count() or 1
    with concurrent.futures.ThreadPoolExecutor(jobs) as pool:
        objs = list(pool.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    subprocess.run([nvcc, *NVCC_FLAGS, "-shared", *objs, "-o", tmp],
                   check=True)
    os.replace(tmp, LIB)
    _build_binding_if_possible(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
