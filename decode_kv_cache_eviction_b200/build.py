"""Build ``librkv.so`` (the C-ABI engine) in-tree for sm_100a with nvcc, and with the host
compiler ``_tensors.so``, the Python binding's argument check.

Usage: ``python -m decode_kv_cache_eviction_b200.build [--force] [--verbose]``.
The shared library is placed next to this file so that it travels with the
source tree.  cudart is linked statically; the CUDA driver entry point for
tensor-map encoding is looked up at run time, so the library loads (and its
host-side checks run) on a machine without a GPU.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "librkv.so")
TENSORS = os.path.join(HERE, "_tensors.so")
TENSORS_SRC = os.path.join(CSRC, "tensors.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared", "--threads", "0",
]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, out: str, verbose: bool):
    """Run a compiler that writes ``out`` (by way of a temporary file)."""
    tmp = out + ".tmp"
    res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed building {os.path.basename(out)}")
    os.replace(tmp, out)


def _built_for() -> str:
    """What _tensors.so depends on beside its source: PyTorch's C++ interface differs between
    versions.  The text is part of the module, which loads into nothing else."""
    import torch
    return f"PyTorch {torch.__version__}, {sys.implementation.cache_tag}"


def _tensors_stale() -> bool:
    if not os.path.exists(TENSORS) or os.path.getmtime(TENSORS) < os.path.getmtime(TENSORS_SRC):
        return True
    with open(TENSORS, "rb") as f:
        return _built_for().encode() + b"\0" not in f.read()


def _build_tensors(verbose: bool):
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
          f'-DRKV_BUILT_FOR="{_built_for()}"',
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(x for i in inc for x in ("-isystem", i)), TENSORS_SRC,
          "-L", os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"],
         TENSORS, verbose)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _tensors_stale():
        _build_tensors(verbose)
    if not force and not _stale():
        return LIB
    cmd = [nvcc_path(), *NVCC_FLAGS, "-I", INCLUDE]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    _run([*cmd, *sources()], LIB, verbose)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
