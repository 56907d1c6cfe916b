"""What the operators between the FP8 products launch, on the CPU: builds
tests/sanitize/layer_launches.cpp with their host code (sanitizers on) and queries it."""
import atexit
import functools
import os
import shutil
import subprocess
import tempfile
from collections import namedtuple
from concurrent.futures import ThreadPoolExecutor

import pytest

from _mx_launches import AVAILABLE, CLANG, CSRC, HIPCC, ROOT, SAN, _run

pytestmark = pytest.mark.skipif(not AVAILABLE, reason="no ROCm toolchain")

Launch = namedtuple("Launch", "kernel grid threads")
DENSE, CONTIGUOUS, MASKED = range(3)
BIG = 0x7fffff00


@functools.lru_cache(None)
def _build():
    tmp = tempfile.mkdtemp(prefix="layer_launches")
    atexit.register(shutil.rmtree, tmp, True)
    sources = [os.path.join(CSRC, f) for f in ("fp8bs_norm.hip", "fp8bs_dispatch.hip", "fp8bs_gated.hip")]
    sources.append(os.path.join(ROOT, "tests", "sanitize", "layer_launches.cpp"))

    def compile_one(src):
        out = os.path.join(tmp, os.path.basename(src) + ".o")
        # the host pass only: no code for the GPU is built here
        _run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g",
              "-std=c++17", "-fno-omit-frame-pointer"] +
             [x for f in SAN for x in ("-Xarch_host", f)] +
             ["-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-c", src, "-o", out])
        return out
    with ThreadPoolExecutor(4) as pool:
        objs = list(pool.map(compile_one, sources))
    # the device code that the host objects would carry
    missing = {line.split()[-1] for line in _run(["nm", "-u"] + objs).splitlines()
               if "__hip_fatbin_" in line}
    exe = os.path.join(tmp, "layer_launches")
    _run([CLANG] + SAN + objs + [f"-Wl,--defsym,{s}=0" for s in sorted(missing)] + ["-o", exe])
    return exe


ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")


def ask(*queries, cap=0):
    """[(status, launches)] of (op, numbers ...)"""
    text = "".join(f"{cap} {q[0]} {' '.join(str(x) for x in (tuple(q[1:]) + (0,) * 5)[:5])}\n" for q in queries)
    r = subprocess.run([_build()], input=text, capture_output=True, text=True, timeout=600, env=ENV)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr
    out = []
    for line in r.stdout.splitlines():
        head, *rest = line.split("; ")
        out.append((int(head), [Launch(x.rsplit(" ", 2)[0].removeprefix("void "), *(int(v) for v in x.rsplit(" ", 2)[1:]))
                                for x in rest]))
    assert len(out) == len(queries)
    return out


F32, BF16, NONE = 0, 1, 2


def types(x, res, weight):
    return x + 4 * res + 16 * weight


# the sizes of the GPU tests (tests/test_gpu_layer_*.py)
NORM = [(1, 128), (3, 384), (1, 2048), (2, 7168), (2, 9088), (3, 16384), (2, 32768), (512, 128), (513, 1024),
        (517, 2048), (512, 2176), (520, 7168), (512, 8320), (513, 16512), (515, 4096), (530, 264), (7, 1000), (1030, 7168)]


def test_every_kernel_is_reached():
    queries = [("norm", r, k, types(x, res, w), 1) for r, k in NORM for x in (F32, BF16)
               for res in (F32, BF16, NONE) for w in (F32, BF16)]
    queries += [("norm_back", r, k, types(s, g, w), 1) for r, k in NORM for s in (F32, BF16)
                for g in (F32, BF16) for w in (F32, BF16)]
    queries += [("dispatch", CONTIGUOUS, t, 8, g, 128 * 4096) for t, g in ((10, 8), (200, 8), (400, 64), (5000, 8), (40000, 8))]
    queries += [("combine", 10, 2, 512, y) for y in (F32, BF16)] + [("combine_back", 10, 2, 512, y) for y in (F32, BF16)]
    queries += [("gated", DENSE, 100, 256, 1, keep + 2 * act) for keep in (0, 1) for act in (0, 1)]
    queries += [("gated_back", m, 256, kept, act) for m in (100, 20000) for kept in (0, 1) for act in (0, 1)]
    queries += [("columns", 100, 256, t) for t in (0, 1, 2)]
    # (inputs read past the caches: tests/test_gpu_layer_large.py)
    queries += [(op, 5000, 3, 4096, y) for op in ("combine", "combine_back") for y in (F32, BF16)]
    queries += [("gated", DENSE, 15000, 1152, 1, keep + 2 * act) for keep in (0, 1) for act in (0, 1)]
    queries += [("columns", 12345, 4096, t) for t in (0, 1, 2)]
    seen = set()
    for q, (st, launches) in zip(queries, ask(*queries)):
        assert st == 0 and launches, q
        seen |= {x.kernel for x in launches}
    out = subprocess.run([_build(), "list"], capture_output=True, text=True, check=True, env=ENV)
    kernels = {line.removeprefix("void ") for line in out.stdout.splitlines()}
    assert kernels == seen, kernels ^ seen


# workgroups that share a CU
SHARE = {"rms_norm_kernel": {256: 8, 1024: 2}, "rms_norm_backward_kernel": {256: 4, 1024: 1},
         "rms_norm_sum_kernel": {1024: 2}, "dispatch_few_kernel": {256: 4}, "dispatch_count_kernel": {256: 4},
         "dispatch_rank_kernel": {256: 4}, "dispatch_rows_kernel": {256: 8}, "combine_kernel": {256: 8},
         "combine_backward_kernel": {256: 8}, "gated_quant_kernel": {256: 8}, "gated_backward_kernel": {1024: 1},
         "quant_128x1_kernel": {512: 4}}


def test_every_launch_keeps_to_the_cap():
    calls = [("norm", 5000, 7168, types(1, 1, 1), 3), ("norm", 300, 7168, types(1, 1, 1), 3), ("norm", 5000, 512, types(1, 1, 1), 3),
             ("norm_back", 5000, 7168, types(1, 1, 1), 1), ("norm_back", 100, 30000, types(1, 1, 1), 1),
             ("dispatch", CONTIGUOUS, 100, 8, 8, 4096), ("dispatch", MASKED, 40000, 8, 256, 3000),
             ("dispatch", CONTIGUOUS, 0, 8, 8, 128 * 9999), ("combine", 5000, 8, 7168, 1),
             ("combine_back", 5000, 8, 7168, 1), ("gated", MASKED, 300, 2048, 16, 1),
             ("gated_back", 5000, 2048, 1, 0), ("columns", 5000, 7168, 1)]
    seen = set()
    for cap in (1, 7, 64):
        for call, (st, launches) in zip(calls, ask(*calls, cap=cap)):
            assert st == 0, call
            for x in launches:
                name = x.kernel.split("<")[0]
                assert 1 <= x.grid <= cap * SHARE[name][x.threads], (call, cap, x)
                seen.add(name)
    assert seen == set(SHARE)


def test_the_cap_does_not_choose_the_order_of_sums():
    """parts of dweight: one a unit, the same units whatever the cap"""
    for rows, k in ((100, 512), (5000, 512), (5000, 7168), (600, 30000)):
        kernels = [[x.kernel for x in ask(("norm_back", rows, k, types(1, 1, 1), 1), cap=cap)[0][1]]
                   for cap in (0, 1, 100)]
        assert kernels[0] == kernels[1] == kernels[2]


def test_large_sizes_are_refused_or_launched_right():
    # (the host code runs with overflow checks, the stand-in refuses grids as HIP does)
    calls = [("norm", BIG, 8, types(1, 1, 1), 1), ("norm", BIG, 32768, types(0, 0, 0), 3),
             ("norm_back", BIG, 32768, types(1, 1, 1), 1), ("dispatch", MASKED, 1 << 24, 64, 1024, BIG // 1024),
             ("dispatch", CONTIGUOUS, 1 << 24, 64, 1024, BIG // 128 * 128), ("dispatch", CONTIGUOUS, 0, 1, 1, BIG // 128 * 128),
             ("dispatch", MASKED, 1, 1, 1024, BIG // 1024), ("combine", 1 << 30, 1, 8), ("combine", 1 << 24, 64, 1 << 24),
             ("combine_back", 1 << 30, 1, 8), ("combine_back", 1 << 24, 64, 1 << 24), ("gated", DENSE, BIG, 128, 1, 1),
             ("gated", MASKED, 1, 128, BIG, 1), ("gated", MASKED, BIG, 1 << 20, BIG, 1), ("gated_back", BIG, 1 << 20, 1, 0),
             ("gated_back", BIG, 128, 1, 0), ("columns", BIG, 1 << 20, 1), ("columns", BIG, 16, 1)]
    launched = 0
    for call, (st, launches) in zip(calls, ask(*calls)):
        assert st in (0, 3), (call, st)
        assert (st == 0) == bool(launches), call
        launched += bool(launches)
    assert launched >= 12
