"""Build libfp8bs.so (HIP for gfx950) in-tree with hipcc, and, where torch is installed, the CPython
module through which the layer operators' small calls reach it (host code alone, with the host
compiler and torch's headers).

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


def _module() -> str | None:
    """The CPython module; None without torch, whose headers it takes."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    torch = os.path.dirname(spec.origin)
    include = os.path.join(torch, "include")
    tmp = MODULE + ".tmp"
    # (hipcc, which the library needs anyway, where there is no other compiler)
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++") or HIPCC
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared",
           "-I" + os.path.join(ROOT, "include"), "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "fp8bs_layer_py.cpp"),
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"fp8bs_layer_py.cpp: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for fp8bs_layer_py.cpp:\n{r.stderr}")
    return tmp


def build(verbose: bool = False) -> str:
    """The library, then the module.  The library needs hipcc alone, and is in place whatever becomes
    of the module: without torch there is none, and a failure of its own is raised last."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        module = ex.submit(_module)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    if os.path.exists(MODULE):                      # (an older one need not fit the library)
        os.remove(MODULE)
    os.replace(tmp, LIB)
    made = module.result()
    if made:
        os.replace(made, MODULE)
    if verbose:
        print(f"built {LIB}" + (f" and {MODULE}" if made else "; no module for the binding without torch"))
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
