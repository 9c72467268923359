"""Build the CUDA library ``_build/libmoe_gb300.so`` in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` compiles to an object in parallel (one ``-gencode``), then nvcc links the shared
library with the static CUDA runtime.  ``csrc/operands.cpp``, the binding's quick argument check, becomes a
Python module beside it (g++ with torch's headers; the library does not need it).  A rebuild happens only when a source or header is newer than
the library.  Usage: ``python -m mixture_experts_ffn_gemm_gb300.build [--force] [--verbose]``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmoe_gb300.so")
OPERANDS_SRC = os.path.join(CSRC, "operands.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the MoE library")


def _inputs():
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(ROOT, "include", "moe.h")]
    return srcs, deps


def _compile(nvcc: str, src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _stale(target: str, deps) -> bool:
    return not os.path.exists(target) or \
        os.path.getmtime(target) < max(os.path.getmtime(p) for p in deps)


def operands_path() -> str:
    """The module of the quick argument check.  It reads tensors by the layout of the torch and the Python that it
    was compiled with, so its name holds both: another version has a module of its own."""
    import torch
    return os.path.join(BUILD, f"_operands.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def build_operands(force: bool = False) -> str:
    """Compile the Python module of the quick argument check; returns its path."""
    target = operands_path()
    if not force and not _stale(target, [OPERANDS_SRC]):
        return target
    import torch
    os.makedirs(BUILD, exist_ok=True)
    home = os.path.dirname(torch.__file__)
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    tmp = target + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{p}" for p in inc], OPERANDS_SRC, "-o", tmp, f"-L{os.path.join(home, 'lib')}",
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for operands.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, target)
    return target


def _try_operands(force: bool = False) -> None:
    """build_operands where there are a C++ compiler and torch's and Python's headers; without them the binding
    makes the same checks in Python."""
    try:
        build_operands(force)
    except (RuntimeError, OSError) as e:
        target = operands_path()
        if os.path.exists(target):  # of older sources
            os.remove(target)
        warnings.warn(f"the quick argument check is not built, calls of the products and microscaled operators "
                      f"check their operands in Python (some 5 us a call more): {e}", RuntimeWarning)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile and link the library; returns its path."""
    srcs, deps = _inputs()
    if not force and not _stale(LIB, deps):
        _try_operands()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        operands = ex.submit(_try_operands, force)
        objs = list(ex.map(lambda s: _compile(nvcc, s, verbose, list(extra)), srcs))
        operands.result()
    tmp = LIB + f".tmp{os.getpid()}"
    # every symbol resolved at link time: a missing definition fails here, not at load time
    r = subprocess.run([nvcc, *ARCH, "-shared", "-Xlinker", "--no-undefined", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas resource usage")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
