"""Build libdilattn.so (nvcc, sm_100a) and the binding's _torch_calls.so (g++) in-tree.

    python -m sparse_long_sequence_dilated_b200.build [--ptxas-v]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "dilattn.cu")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdilattn.so")
CALLS_SRC = os.path.join(PKG, "csrc", "torch_calls.cpp")
CALLS = os.path.join(PKG, "_torch_calls.so")


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def build(ptxas_verbose: bool = False, out: str = LIB) -> str:
    cmd = [
        nvcc_path(), "-O3", "-std=c++17",
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-lineinfo", "-shared", "-Xcompiler", "-fPIC,-O3", "-cudart", "static",
        "-I", INCLUDE, "-I", os.path.join(PKG, "csrc"),
        "-o", out, SRC,
    ]
    if ptxas_verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if ptxas_verbose:
        sys.stderr.write(res.stderr)
    return out


def build_calls(out: str = CALLS) -> str:
    """The binding's compiled calls, against this interpreter's torch (whose libraries are
    loaded before it)."""
    import sysconfig

    import torch

    top = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    cmd = [
        shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-I", INCLUDE, "-I", os.path.join(top, "include"),
        "-I", os.path.join(top, "include", "torch", "csrc", "api", "include"),
        "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
        "-o", out, CALLS_SRC, "-L", os.path.join(top, "lib"),
        "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
    ]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return out


if __name__ == "__main__":
    build(ptxas_verbose="--ptxas-v" in sys.argv)
    build_calls()
    print(LIB)
