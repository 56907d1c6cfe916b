"""The order in which the norm's backward pass adds dweight over rows follows from the sizes alone: on
the CPU, tests/sanitize/norm_sums.cpp (host code, sanitizers on) tells in which parts a launch adds, under
several caps on CUs and on devices of several sizes."""
import atexit
import functools
import os
import shutil
import subprocess
import tempfile

import pytest

from _mx_launches import AVAILABLE, CLANG, CSRC, HIPCC, ROOT, SAN, _run

pytestmark = pytest.mark.skipif(not AVAILABLE, reason="no ROCm toolchain")


@functools.lru_cache(None)
def _build():
    tmp = tempfile.mkdtemp(prefix="norm_sums")
    atexit.register(shutil.rmtree, tmp, True)
    obj, exe = os.path.join(tmp, "norm_sums.o"), os.path.join(tmp, "norm_sums")
    # the host pass only: no code for the GPU is built here
    _run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17",
          "-fno-omit-frame-pointer"] + [x for f in SAN for x in ("-Xarch_host", f)] +
         ["-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-c",
          os.path.join(ROOT, "tests", "sanitize", "norm_sums.cpp"), "-o", obj])
    missing = {line.split()[-1] for line in _run(["nm", "-u", obj]).splitlines() if "__hip_fatbin_" in line}
    _run([CLANG] + SAN + [obj] + [f"-Wl,--defsym,{s}=0" for s in sorted(missing)] + ["-o", exe])
    return exe


def launches(queries):
    """[[(grid, kernel, numbers ...)]] of (cap, CUs, rows, k, in place)"""
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    text = "".join(" ".join(str(int(x)) for x in q) + "\n" for q in queries)
    r = subprocess.run([_build()], input=text, capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr
    out = []
    for line in r.stdout.splitlines():
        status, *rest = line.split("; ")
        assert status == "0", line
        out.append([(int(g), kernel, *map(int, numbers)) for g, kernel, *numbers in (x.split(" ") for x in rest)])
    assert len(out) == len(queries)
    return out


ROWS = [1, 5, 64, 383, 384, 385, 512, 600, 1024, 1025, 2047, 2048, 5000, 100000]
COLUMNS = [8, 512, 1000, 2048, 4096, 7168, 8192, 16384, 32768]
MACHINES = [(0, 256), (1, 256), (7, 256), (64, 256), (256, 256), (1000, 256), (0, 304), (0, 64), (40, 64)]


def test_parts_of_dweight_follow_from_the_sizes():
    sizes = [(rows, k, in_place) for rows in ROWS for k in COLUMNS for in_place in (0, 1)]
    runs = [launches([(cap, cus, *size) for size in sizes]) for cap, cus in MACHINES]
    grids = set()
    for i, (rows, k, in_place) in enumerate(sizes):
        kinds = {tuple(x[1:] for x in run[i]) for run in runs}
        assert len(kinds) == 1, (rows, k, in_place, kinds)
        kind = kinds.pop()
        if rows <= 384:                            # straight from the inputs, rows and columns apart if in place
            tiles = (k + 63) // 64
            assert sum(x[2] for x in kind) == tiles and all(x[0] == "rows" and x[3] for x in kind), kind
            assert len(kind) == 1 + in_place
        else:                                      # a part a unit, all of them added
            (_, units, none, direct), (kernel, parts, _) = kind
            assert kernel == "sum" and parts == units and none == direct == 0, kind
            assert units <= 512
        grids.add(tuple(run[i][0][0] for run in runs))
    # (the machines do differ in what they launch)
    assert any(len(set(g)) > 3 for g in grids)
