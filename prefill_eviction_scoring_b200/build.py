"""Build libwaits.so in-tree with nvcc for sm_100a (no JIT, no cache dir), and
the Python binding of the cache operators with g++ against torch's headers.

``python -m prefill_eviction_scoring_b200.build`` compiles every ``csrc/*.cu``
into ``prefill_eviction_scoring_b200/libwaits.so`` and
``csrc/torch/binding.cpp`` into ``prefill_eviction_scoring_b200/_binding.so``;
each is left alone when it is newer than its sources and headers.
"""

from __future__ import annotations

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
LIB = os.path.join(PKG, "libwaits.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "torch", "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin on PATH)")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps)


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _stale():
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + res.stdout + res.stderr)
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """``_binding.so``, linked to the libwaits.so beside it."""
    if not force and not _older(BINDING, [BINDING_SRC] + _headers()):
        return BINDING
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = cpp_extension.include_paths() + [os.path.join(cuda, "include"),
                                           sysconfig.get_paths()["include"], INCLUDE]
    tmp = BINDING + ".tmp"
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    _run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f"-isystem{p}" for p in inc), BINDING_SRC, "-o", tmp,
          *(f"-L{p}" for p in cpp_extension.library_paths()), f"-L{PKG}", "-l:libwaits.so",
          "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
          "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if force or _stale():
        tmp = LIB + ".tmp"
        _run([_nvcc(), *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-o", tmp, *sources()],
             verbose)
        os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
