"""What the MXFP4 entry points launch for given sizes, asked on the CPU: builds
tests/sanitize/mx_launches.cpp with the operators' host code (sanitizers on) and queries it."""
import atexit
import functools
import os
import shutil
import subprocess
import tempfile
from collections import namedtuple
from concurrent.futures import ThreadPoolExecutor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_grouped_gemm_block_amd", "csrc")
SAN = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all"]
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang++"
AVAILABLE = os.path.exists(HIPCC) and os.path.exists(CLANG)

DENSE, CONTIGUOUS, MASKED = range(3)
Launch = namedtuple("Launch", "kernel args grid threads")
Result = namedtuple("Result", "status launches")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return r.stdout


@functools.lru_cache(None)
def _build():
    tmp = tempfile.mkdtemp(prefix="mx_launches")
    atexit.register(shutil.rmtree, tmp, True)
    sources = [os.path.join(CSRC, f) for f in (
        "fp8bs_mx_api.cpp", "fp8bs_mx_gemm.hip", "fp8bs_mx_stream.hip", "fp8bs_mx_grad.hip",
        "fp8bs_mx_quant.hip")] + [os.path.join(ROOT, "tests", "sanitize", "mx_launches.cpp")]

    def compile_one(src):
        out = os.path.join(tmp, os.path.basename(src) + ".o")
        # the host pass only: no code for the GPU is built here
        _run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g",
              "-std=c++17", "-fno-omit-frame-pointer"] +
             [x for f in SAN for x in ("-Xarch_host", f)] +
             ["-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-c", src, "-o", out])
        return out
    with ThreadPoolExecutor(6) as pool:
        objs = list(pool.map(compile_one, sources))
    # the device code that the host objects would carry
    missing = {line.split()[-1] for line in _run(["nm", "-u"] + objs).splitlines()
               if "__hip_fatbin_" in line}
    exe = os.path.join(tmp, "mx_launches")
    _run([CLANG] + SAN + objs + [f"-Wl,--defsym,{s}=0" for s in sorted(missing)] + ["-o", exe])
    return exe


def _kernel(name):
    """(name, template arguments) of a kernel"""
    kernel, _, args = name.removeprefix("void ").partition("<")
    args = tuple(int(x) if x.strip().lstrip("-").isdigit() else x.strip() == "true"
                 for x in args.rstrip("> ").split(",")) if args else ()
    return kernel, args


def instances():
    """every compiled kernel of the operators"""
    out = subprocess.run([_build(), "list"], capture_output=True, text=True, check=True,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    return {_kernel(line) for line in out.stdout.splitlines()}


def ask(queries):
    """[Result] of [(op, layout, m, expected, n, k, groups, flag, cap)], the last ones optional"""
    lines = []
    for q in queries:
        op, layout, m, expected, n, k, groups, flag, cap = (tuple(q) + (1, 0, 0)[len(q) - 6:])[:9]
        lines.append(f"{cap} {op} {layout} {m} {expected} {n} {k} {groups} {flag}\n")
    r = subprocess.run([_build()], input="".join(lines), capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0",
                                UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr
    out = []
    for line in r.stdout.splitlines():
        head, *rest = line.split("; ")
        launches = []
        for part in rest:
            name, grid, threads = part.rsplit(" ", 2)
            launches.append(Launch(*_kernel(name), int(grid), int(threads)))
        out.append(Result(int(head), launches))
    assert len(out) == len(lines)
    return out
