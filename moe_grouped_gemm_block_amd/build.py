"""Build libfp8bs.so (HIP for gfx950) in-tree with hipcc, and the CPython module through which
the layer operators' small calls reach it (host code alone, with the host compiler and torch's
headers).

    python -m moe_grouped_gemm_block_amd.build

Every HIP translation unit is compiled with packed FP32 instructions disabled
(``-Xclang -target-feature -Xclang -packed-fp32-ops``); the host pass warns
that it does not know that feature, which is harmless.  The device pass also
schedules with the AMDGPU register-pressure trackers (see DEVICE below).
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libfp8bs.so")
MODULE = os.path.join(LIBDIR, "fp8bs_layer_py.so")
BUILD_DIR = os.path.join(ROOT, "_build")
ARCH = os.environ.get("FP8BS_OFFLOAD_ARCH", "gfx950")

SOURCES = ["fp8bs_gemm.hip", "fp8bs_quant.hip", "fp8bs_api.cpp", "fp8bs_planner.cpp",
           "fp8bs_mx_gemm.hip", "fp8bs_mx_stream.hip", "fp8bs_mx_grad.hip",
           "fp8bs_mx_quant.hip", "fp8bs_mx_api.cpp",
           "fp8bs_norm.hip", "fp8bs_dispatch.hip", "fp8bs_gated.hip"]
HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")

COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
          "-I" + os.path.join(ROOT, "include")]
# -amdgpu-use-amdgpu-trackers: the machine scheduler tracks register pressure with the
# AMDGPU-specific trackers; same-machine A/B runs (traced, cold) measured the MoE contiguous
# shapes 2-3% faster with it and every other family within +-1% (same register counts for
# the dense and contiguous 256x256 kernels, a different instruction order).
DEVICE = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-munsafe-fp-atomics", "-mllvm", "-amdgpu-use-amdgpu-trackers"]


def _compile(src: str) -> str:
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD_DIR, src + ".o")
    cmd = [HIPCC, "-x", "hip"] + DEVICE + COMMON + ["-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _module() -> str:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    include = os.path.join(torch, "include")
    tmp = MODULE + ".tmp"
    cmd = [os.environ.get("CXX", shutil.which("g++") or "c++"), "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared",
           "-I" + os.path.join(ROOT, "include"), "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "fp8bs_layer_py.cpp"),
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for fp8bs_layer_py.cpp:\n{r.stderr}")
    os.replace(tmp, MODULE)
    return MODULE


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        module = ex.submit(_module)
        objs = list(ex.map(_compile, SOURCES))
        module.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB} and {MODULE}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
