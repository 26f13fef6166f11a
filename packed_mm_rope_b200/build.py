"""Build libh3.so in-tree for sm_100a with nvcc, and its tensor binding with the host compiler.

    python -m packed_mm_rope_b200.build          # or build_library()

The library is one translation unit (csrc/h3.cu includes the kernels), linked
against the static CUDA runtime; the driver's tensor-map encoder is looked up
at run time, so no libcuda link is needed.  _tensors.so (csrc/binding.cpp) is a
Python module over the library's C ABI, linked against it and PyTorch; where there
is no PyTorch with CUDA to build it against, the library is built alone.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libh3.so")
CSRC = os.path.join(HERE, "csrc")
HEADER = os.path.join(ROOT, "include", "h3.h")
BINDING = os.path.join(HERE, "_tensors.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")


def sources() -> list:
    """Every file the library is built from: all of csrc/ and the public header."""
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + [HEADER]


NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-v",
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date(target: str = LIB) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    made_from = sources() if target == LIB else [BINDING_SOURCE, HEADER]
    return all(os.path.getmtime(s) <= t for s in made_from + [__file__])


def _run(cmd: list, target: str, verbose: bool) -> None:
    r = subprocess.run(cmd + ["-o", target + ".tmp"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + r.stdout + r.stderr)
    os.replace(target + ".tmp", target)
    if verbose:
        sys.stdout.write(r.stderr)


def _cxx():
    return shutil.which("g++") or shutil.which("c++")


def binding_lacks() -> str | None:
    """What the tensor binding would need and is not there, or None."""
    try:
        import torch
    except ImportError:
        return "PyTorch"
    if torch.version.cuda is None:
        return "a PyTorch with CUDA"
    if _cxx() is None:
        return "a C++ compiler"
    if not os.path.exists(os.path.join(sysconfig.get_path("include"), "Python.h")):
        return "the Python headers"
    return None


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Build _tensors.so; raises RuntimeError where that cannot be done."""
    if not force and up_to_date(BINDING):
        return BINDING
    lacks = binding_lacks()
    if lacks is not None:
        raise RuntimeError(f"{os.path.basename(BINDING)} cannot be built without {lacks}")
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [sysconfig.get_path("include"), *cpp_extension.include_paths(), os.path.join(cuda, "include")]
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-DNDEBUG",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for path in include:
        cmd += ["-isystem", path]
    cmd += [BINDING_SOURCE, "-L", HERE, "-lh3", "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
            "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    _run(cmd, BINDING, verbose)
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build libh3.so and, where it can be built, the tensor binding; returns the library's path.

    A user of the C ABI needs no PyTorch: without one the binding is left out, with a line on stderr, and
    the Python calls that go through it raise ImportError.
    """
    if force or not up_to_date():
        _run([nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, "h3.cu")], LIB, verbose)
    if force or not up_to_date(BINDING):
        lacks = binding_lacks()
        if lacks is not None:
            sys.stderr.write(f"{os.path.basename(BINDING)} left out: no {lacks.removeprefix('a ')}\n")
            return LIB
        build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose=True)
    print(LIB)
