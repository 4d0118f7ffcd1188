"""Builds libsgq.so in-tree with nvcc for sm_100a (B200).

    python -m activation_sparse_quantized_b200.build [--force] [--verbose]

nvcc cross-compiles without a GPU. The library is linked against the static
CUDA runtime so that it does not depend on which libcudart the Python process
loaded first.
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libsgq.so")
BINDING_SOURCE = os.path.join(CSRC, "tensors.cpp")
BINDING_PATH = os.path.join(PKG, "_tensors.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=default", "-shared", "-cudart", "static",
         "--threads", "0"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def build_binding(force: bool = False) -> str:
    """Compile the binding's helper module (if stale) against this Python and torch."""
    if not force and os.path.exists(BINDING_PATH) and os.path.getmtime(BINDING_PATH) >= max(
            os.path.getmtime(p) for p in (BINDING_SOURCE, __file__)):
        return BINDING_PATH
    import torch
    at = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(at, "include"),
           "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"), BINDING_SOURCE, "-o", BINDING_PATH + ".tmp",
           "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    subprocess.run(cmd, check=True)
    os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
    return BINDING_PATH


def is_stale(out: str = LIB_PATH) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in sources() + headers() + [__file__])


def build(force: bool = False, verbose: bool = False, out: str = LIB_PATH) -> str:
    """Compile every .cu under csrc/ into one shared library (if stale), and the binding's helper."""
    if out == LIB_PATH:
        build_binding(force)
    if not force and not is_stale(out):
        return out
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", INCLUDE, *sources(), "-o", out + ".tmp"]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)
    return out


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/smem usage")
    a = ap.parse_args(argv)
    print(build(force=a.force or a.verbose, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
