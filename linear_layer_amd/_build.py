"""Build liblinear_layer.so (the C-ABI library) for gfx950 with hipcc, and the Python
module _call.so on top of it where torch is installed, in-tree.

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


def _build_call() -> bool:
    """The module that takes tensors apart for the short calls (csrc/call.cpp), with hipcc
    as the host's compiler; False where there is no torch, which the C library and its
    users do without."""
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return False
    torch = os.path.dirname(spec.origin)
    tmp = CALL + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           os.path.join(CSRC, "call.cpp"), "-x", "none", "-o", tmp, "-I", INCLUDE, "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-L", PKG, "-l:liblinear_layer.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-Wl,-rpath," + os.path.join(torch, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building _call.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)
    return True


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
    call = _build_call()
    if verbose:
        print("built", LIB)
        print("built " + CALL if call else "no torch: without " + CALL)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
