"""Build liblinear_layer.so (the C-ABI library) for gfx950 with hipcc, and the Python
module _call.so on top of it with the host compiler, in-tree.

Usage: ``python -m linear_layer_amd._build``. Cross-compiles without a GPU.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblinear_layer.so")
CALL = os.path.join(PKG, "_call.so")
OBJDIR = os.path.join(PKG, "_build")

SOURCES = ["api.hip", "gemm_f32.hip", "gemm_f32_nt.hip", "gemm_f16.hip", "elementwise.hip",
           "api_mx4.hip", "mx4.hip", "gemm_mx4.hip", "gemm_mx4_tile.hip", "api_norm.hip", "rmsnorm.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # keep the compiler from forming packed-FP32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_call() -> None:
    """The module that takes tensors apart for the short calls (csrc/call.cpp)."""
    import importlib.util
    import sysconfig
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    tmp = CALL + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           os.path.join(CSRC, "call.cpp"), "-o", tmp, "-I", INCLUDE, "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-L", PKG, "-l:liblinear_layer.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-Wl,-rpath," + os.path.join(torch, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building _call.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    jobs = min(len(SOURCES), os.cpu_count() or 4, 16)
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _build_call()
    if verbose:
        print("built", LIB)
        print("built", CALL)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
