"""Which kernels the MXFP4 entry points launch, on the CPU (tests/_mx_launches.py)."""
import pytest

from _mx_cases import CASES
from _mx_launches import AVAILABLE, CONTIGUOUS, DENSE, MASKED, ask, instances

pytestmark = pytest.mark.skipif(not AVAILABLE, reason="no ROCm toolchain")

# m (rows of a slot), n (f), k, groups
SLOTS = [(256, 7168, 2048, 4), (256, 7168, 2048, 16), (16, 7168, 2048, 16), (256, 2048, 7168, 2),
         (256, 2048, 7168, 8), (64, 2048, 7168, 16), (1024, 2048, 7168, 8), (300, 256, 384, 5),
         (4096, 512, 1024, 32), (1, 128, 128, 1)]
ROWS = [(1, 4096, 7168), (64, 4096, 7168), (256, 7168, 2048), (512, 4096, 7168), (600, 2048, 512),
        (4096, 7168, 2048), (200, 416, 640)]


def sums(result):
    """the kernels whose order of summation differs, as launched; dense, the few-rows kernel's
    with its tile (the number of wavefronts that share K follows from it)"""
    assert result.status == 0
    return [(x.kernel, x.args[:2] if x.kernel == "mx_stream_kernel" and x.args[2] == DENSE else None)
            for x in result.launches if x.kernel in ("mx_stream_kernel", "mx_gemm_kernel")]


@pytest.mark.parametrize("op", ["product", "gated", "gated_q", "layer"])
def test_neither_hint_nor_cap_chooses_the_order_of_sums(op):
    # include/fp8bs.h: expected_m "never changes results", nor does the cap on CUs
    for m, n, k, g in SLOTS:
        runs = [(op, MASKED, m, e, n, k, g, 256, cap) for cap in (0, 200, 64, 1)
                for e in (0, 1, 16, 40, 65, 200, m, 2 * m)]
        got = [sums(r) for r in ask(runs)]
        assert all(x == got[0] for x in got), (m, n, k, g)
    for m, n, k in ROWS:
        if op in ("gated_q", "layer"):
            n = n // 128 * 128
        got = [sums(r) for r in ask([(op, DENSE, m, 0, n, k, 1, 256, cap) for cap in (0, 255, 64, 8, 1)])]
        assert all(x == got[0] for x in got), (m, n, k)


@pytest.mark.parametrize("layout", [DENSE, CONTIGUOUS])
def test_the_cap_does_not_choose_how_gradients_are_summed(layout):
    # the recomputed gate and up projections, and into how many parts a product is split (a
    # launch of the kernel that adds parts; the 128x128 and 256x256 tiles sum alike)
    for m, f, k, g in [(200, 416, 640, 1), (512, 2048, 2048, 4), (2048, 64, 256, 3), (4096, 2048, 7168, 8),
                       (128, 4096, 4096, 2)]:
        m = m if layout == DENSE else (m + 127) // 128 * 128
        for flag in (1, 2, 3, 7, 15):
            got = ask([("backward", layout, m, 0, f, k, g, flag, cap) for cap in (0, 200, 64, 1)])
            for r in got:
                assert sums(r) == sums(got[0])
                assert (sum(x.kernel == "mx_grad_sum_kernel" for x in r.launches) > 0) == (
                    sum(x.kernel == "mx_grad_sum_kernel" for x in got[0].launches) > 0)


# workgroups of a kernel that share a CU (by LDS and threads)
SHARE = {"mx_stream_kernel": 1, "mx_grad_pair_kernel": 2, "mx_grad_sum_kernel": 8, "mx_quant_kernel": 8,
         "mx_dequant_kernel": 8, "mx_block_order_kernel": 1}


def test_every_launch_keeps_to_the_cap():
    calls = [("product", DENSE, 128, 0, 2112, 7168, 1), ("product", DENSE, 4096, 0, 7168, 2048, 1),
             ("product", DENSE, 1, 0, 4096, 7168, 1), ("product", MASKED, 40, 9, 7168, 2048, 9),
             ("gated", MASKED, 256, 16, 2048, 7168, 8), ("gated_q", CONTIGUOUS, 8192, 0, 512, 1024, 3),
             ("layer", DENSE, 64, 0, 2048, 7168, 1, 7168), ("quantise", DENSE, 3000, 0, 0, 7168, 4, 1),
             ("dequantise", DENSE, 3000, 0, 0, 7168, 4, 0), ("backward", DENSE, 200, 0, 416, 640, 1, 3),
             ("backward", DENSE, 16384, 0, 128, 256, 1, 3), ("backward", DENSE, 8192, 0, 512, 1024, 1, 2),
             ("backward", DENSE, 128, 0, 4096, 4096, 1, 1), ("backward", DENSE, 1024, 0, 2048, 2048, 1, 3),
             ("backward", CONTIGUOUS, 2048, 0, 512, 1024, 8, 7),
             ("backward", CONTIGUOUS, 16384, 0, 2048, 7168, 8, 3)]
    seen = set()
    for cap in (1, 7, 64):
        for call, r in zip(calls, ask([(c + (0,) * (8 - len(c)) + (cap,)) for c in calls])):
            assert r.status == 0, call
            for x in r.launches:
                per_cu = SHARE.get(x.kernel) or (1 if x.args[0] == 256 else 2)
                assert 1 <= x.grid <= cap * per_cu, (call, cap, x)
                seen.add(x.kernel)
    assert seen == set(SHARE) | {"mx_gemm_kernel", "mx_grad_kernel"}


def test_no_launch_has_more_threads_than_a_32_bit_number():
    # (the stand-in for the launch refuses such a grid, as HIP does)
    calls = [("quantise", DENSE, 1, 0, 0, 128, 20_000_000, 1), ("quantise", DENSE, 600_000_000, 0, 0, 128, 1, 1),
             ("dequantise", DENSE, 1, 0, 0, 128, 20_000_000), ("product", MASKED, 1, 0, 16, 128, 10_000_000),
             ("product", DENSE, 1, 0, 1 << 29, 128, 1), ("gated", MASKED, 1, 0, 32, 128, 30_000_000),
             ("backward", DENSE, 1 << 29, 0, 32, 128, 1, 3)]
    for call, r in zip(calls, ask(calls)):
        assert r.status == 0, (call, r)
        assert all(x.grid * x.threads < 1 << 32 for x in r.launches), (call, r)


def test_the_cases_compared_on_the_gpu_launch_every_kernel():
    seen = {}
    for case, r in zip(CASES, ask(CASES)):
        assert r.status == 0, case
        for x in r.launches:
            seen.setdefault((x.kernel, x.args), []).append((case, x))
    assert not instances() - set(seen)
    # 256x256 tiles: also more of them than workgroups, and lists longer than a launch takes
    for layout in (DENSE, CONTIGUOUS, MASKED):
        for epilogue in (0, 2, 3):
            assert any(x.grid == 256 for _, x in seen["mx_gemm_kernel", (256, 256, 2, 4, layout, epilogue)])
    for kernel in ("mx_gemm_kernel", (256, 256, 2, 4, MASKED, 0)), ("mx_gemm_kernel", (128, 128, 2, 2, MASKED, 2)):
        cases = [case for case, _ in seen[kernel]]
        assert max(cases.count(c) for c in cases) > 1, kernel


def test_sizes_past_any_memory_are_refused_or_counted_right():
    # (the host code runs with overflow checks here)
    big, wide = 0x7fffffff, 1 << 21
    layer, layer2, call, size, size2 = ask([
        ("layer_size", MASKED, 1 << 20, 0, 1 << 14, 1 << 14, big), ("layer_size", MASKED, 1 << 20, 0, 128, 256, 1 << 12),
        ("layer", MASKED, 1 << 20, 3, 1 << 14, 1 << 14, big, 5),
        ("size", CONTIGUOUS, 1 << 20, 0, wide, 128, 1 << 20, 3), ("size", CONTIGUOUS, 1 << 20, 0, wide, 128, 1, 3)])
    assert layer.status == -1 and call.status == 1 and not call.launches
    assert layer2.status == (1 << 32) * (128 + 64) + (1 << 12) * (2 + 1) * (1 << 20) * 4
    # dg and du of every row, and the blocks by expert; nothing is split
    rows = (1 << 20) * 2 * wide * 2
    assert size.status == rows + ((1 << 20) + 1 + (1 << 13) + 4) * 4
    assert size2.status == rows + (1 + 1 + (1 << 13) + 4) * 4
    refused = [("quantise", DENSE, big, 0, 0, 1 << 24, big, 1), ("product", MASKED, 0x7ffffe00, 5, 1 << 20, 128, big),
               ("gated", MASKED, 0x7ffffe00, 5, 1 << 20, 128, big), ("product", DENSE, 1 << 29, 0, 1 << 29, 128, 1),
               ("backward", DENSE, 1 << 26, 0, 1 << 20, 128, 1, 7)]
    for call, r in zip(refused, ask(refused)):
        assert r.status in (1, 3) and not r.launches, (call, r)
    # more tiles than a 32-bit number counts, of the last of several kernels: refused before the first
    for r in ask([("backward", CONTIGUOUS, 1 << 20, 0, wide, 128, 1 << 20, 3),
                  ("layer", MASKED, 1, 0, 128, 128, 1 << 30, 300)]):
        assert r.status == 3 and not r.launches


def test_of_equal_tiles_the_tallest():
    # 64 rows, 7168 x 2048: 64x32 tiles and 32x64 ones draw as much and are as many rounds; the
    # taller read the weights once (5.2 against 5.6 us)
    (r,) = ask([("product", DENSE, 64, 0, 7168, 2048, 1)])
    assert [x.args for x in r.launches] == [(4, 2, DENSE, 0)]
