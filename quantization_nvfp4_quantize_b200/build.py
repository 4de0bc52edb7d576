"""Build the sm_100a shared library ``libnvfp4_quads.so`` in-tree with nvcc, and
the compiled half of the Python binding (``_binding.so``, host code only) with
g++ against the installed torch's headers.

Every translation unit under ``csrc/`` is compiled for
``-gencode arch=compute_100a,code=sm_100a`` (no other architecture, no
fast-math; the quantization arithmetic relies on IEEE round-to-nearest
intrinsics) and linked into one C-ABI library next to this file.  Objects go to
``_build/`` (git-ignored).  Rebuilds only what changed.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libnvfp4_quads.so")
BINDING = os.path.join(HERE, "_binding.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-std=c++17", "-O3", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if _stale(obj, [src] + _headers()) or verbose_ptxas:
        cmd = [NVCC, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose_ptxas:
            cmd[1:1] = ["-Xptxas", "-v"]
        subprocess.check_call(cmd)
    return obj


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp into the extension module _binding.so."""
    import sysconfig

    import torch
    src = os.path.join(CSRC, "binding.cpp")
    root = os.path.dirname(torch.__file__)
    if force or _stale(BINDING, [src, os.path.join(root, "version.py")] + _headers()):
        tmp = BINDING + ".tmp%d" % os.getpid()
        dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
        subprocess.check_call(["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
                               *[f for d in dirs for f in ("-isystem", d)], src, "-o", tmp,
                               "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
                               "-lc10_cuda", "-lc10"])
        os.replace(tmp, BINDING)
    return BINDING


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    """Compile csrc/*.cu and link libnvfp4_quads.so (returns its path), and
    build the binding.  The library needs nvcc alone: it is linked even where
    the binding cannot be built, whose error is raised at the end."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        binding = ex.submit(build_binding, force)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
        if _stale(LIB, objs):
            tmp = LIB + ".tmp%d" % os.getpid()
            subprocess.check_call([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
                                   "-lcudart"])
            os.replace(tmp, LIB)
        binding.result()
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv, force="--force" in sys.argv))
