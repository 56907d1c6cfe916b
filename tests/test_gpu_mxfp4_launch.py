"""GPU tests of the MXFP4 operators' choice of kernels: what the hint and the cap on compute
units may not change."""
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs

pytestmark = pytest.mark.gpu


def operand(gen, *shape):
    """random codes and exponents of a matrix [.., rows, k]; the exponents lie so far apart that
    sums in 32 bits are rounded (within a few octaves they would be exact in any order)"""
    *lead, rows, k = shape
    q = torch.randint(0, 256, (*lead, rows, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    sf = torch.randint(112, 132, (*lead, k // 128, fp8bs.get_sfa_ld(rows), 4), dtype=torch.uint8,
                       device="cuda", generator=gen).view(torch.int32)[..., 0].contiguous()
    return q, sf


@pytest.fixture
def gen():
    return torch.Generator("cuda").manual_seed(7)


@pytest.fixture
def cap():
    yield fp8bs.set_num_cus
    fp8bs.set_num_cus(0)


# slots, rows of a slot, n (2f), k: the few-rows kernel alone, both by the slots' counts, the
# tiled kernels alone (of 2 x 256 slots' rows as many as the hint says would do)
SLOTS = [(4, 256, 7168, 2048), (16, 60, 512, 1024), (2, 520, 2000, 7168), (8, 256, 4096, 2048),
         (16, 200, 7168, 512)]


@pytest.mark.parametrize("g,max_m,n,k", SLOTS)
def test_the_hint_changes_no_result(gen, g, max_m, n, k):
    a, sfa = operand(gen, g, max_m, k)
    b, sfb = operand(gen, g, n, k)
    masked = torch.tensor([(37 * i + 11) % (max_m + 1) for i in range(g)], dtype=torch.int32, device="cuda")
    masked[-1] = max_m
    runs = []
    for expected in (0, 1, 16, 33, 64, 100, 256, max_m):
        print(f"[gpu] {g} slots {max_m}x{n}x{k} expected {expected}", flush=True)
        d = torch.zeros(g, max_m, n, dtype=torch.bfloat16, device="cuda")
        fp8bs.fp8bs_grouped_masked_nt_mxfp4(a, sfa, b, sfb, d, masked, expected_m=expected)
        outs = [d]
        if n % 256 == 0:
            f = n // 2
            h = torch.zeros(g, max_m, f, dtype=torch.bfloat16, device="cuda")
            fp8bs.fp8bs_gated_masked_mxfp4(a, sfa, b, sfb, h, masked, expected_m=expected)
            hq = torch.zeros(g, max_m, f // 2, dtype=torch.uint8, device="cuda")
            sfh = torch.zeros(g, f // 128, fp8bs.get_sfa_ld(max_m), dtype=torch.int32, device="cuda")
            fp8bs.fp8bs_gated_masked_mxfp4_q(a, sfa, b, sfb, hq, sfh, masked, expected_m=expected)
            outs += [h, hq, sfh]
        runs.append(outs)
    for outs in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs, runs[0]))
    assert runs[0][0][-1].any(-1).all()


@pytest.mark.parametrize("m,n,k", [(256, 7168, 2048), (48, 4096, 7168), (512, 4096, 1024), (700, 2048, 640)])
def test_the_cap_changes_no_result(gen, cap, m, n, k):
    a, sfa = operand(gen, m, k)
    b, sfb = operand(gen, n, k)
    dh = torch.randn(m, n // 2, device="cuda", generator=gen).bfloat16()
    runs = []
    for cus in (0, 255, 64, 9):
        print(f"[gpu] {m}x{n}x{k} cap {cus}", flush=True)
        cap(cus)
        d = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        h = torch.empty(m, n // 2, dtype=torch.bfloat16, device="cuda")
        da = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
        db = torch.empty(n, k, device="cuda")
        fp8bs.fp8bs_dense_nt_mxfp4(a, sfa, b, sfb, d)
        fp8bs.fp8bs_gated_dense_mxfp4(a, sfa, b, sfb, h)
        fp8bs.fp8bs_gated_dense_mxfp4_backward(a, sfa, b, sfb, dh, da, db)
        runs.append((d, h, da, db))
    for outs in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs, runs[0]))


def test_few_workgroups_do_all_of_the_work(gen, cap):
    # each under a cap of 3 CUs against all of them: the quantiser and its inverse, slots, and the
    # gradients side by side and in parts (dense; contiguous with an expert without rows)
    x = torch.randn(3, 301, 1152, device="cuda", generator=gen).bfloat16()
    a, sfa = operand(gen, 5, 70, 640)
    b, sfb = operand(gen, 5, 520, 640)
    masked = torch.tensor([70, 0, 3, 64, 17], dtype=torch.int32, device="cuda")
    layout = torch.tensor([0, 0, 2, 0, 3, 3, 2], dtype=torch.int32, device="cuda").repeat_interleave(128)
    layout[-60:] = -1
    c, sfc = operand(gen, layout.numel(), 384)
    w, sfw = operand(gen, 4, 832, 384)
    long, sfl = operand(gen, 2085, 256)
    v, sfv = operand(gen, 128, 256)
    dh = torch.randn(layout.numel(), 416, device="cuda", generator=gen).bfloat16()
    dl = torch.randn(2085, 64, device="cuda", generator=gen).bfloat16()
    runs = []
    for cus in (0, 3):
        cap(cus)
        print(f"[gpu] cap {cus}", flush=True)
        q, sf = fp8bs.quantize_mxfp4(x)
        sf[..., 301:] = 0                                  # (alignment padding is not written)
        y = fp8bs.dequantize_mxfp4(q, sf, torch.float32)
        d = torch.zeros(5, 70, 520, dtype=torch.bfloat16, device="cuda")
        fp8bs.fp8bs_grouped_masked_nt_mxfp4(a, sfa, b, sfb, d, masked, expected_m=20)
        da = torch.zeros(layout.numel(), 384, dtype=torch.bfloat16, device="cuda")
        db = torch.zeros(4, 832, 384, device="cuda")
        fp8bs.fp8bs_gated_contiguous_mxfp4_backward(c, sfc, w, sfw, dh, da, db, layout)
        ga = torch.zeros(2085, 256, dtype=torch.bfloat16, device="cuda")
        gb = torch.ones(128, 256, device="cuda")
        fp8bs.fp8bs_gated_dense_mxfp4_backward(long, sfl, v, sfv, dl, ga, gb, accumulate=True)
        runs.append((q, sf, y, d, da, db, ga, gb))
    for i, (one, other) in enumerate(zip(*runs)):
        assert torch.equal(one, other), i
        assert one.any()


def test_more_tiles_than_a_launch_has_workgroups(gen):
    # 17 million groups of one row: with a workgroup of 256 threads each, more threads than a
    # launch may have
    g = 17_000_000
    print(f"[gpu] {g} groups", flush=True)
    few = torch.randn(1000, 128, device="cuda", generator=gen).bfloat16()
    x = few.repeat(g // 1000, 1).view(g, 1, 128)
    q, sf = fp8bs.quantize_mxfp4(x)
    want, words = fp8bs.quantize_mxfp4(few)
    assert torch.equal(q.view(g // 1000, 1000, 64), want.expand(g // 1000, 1000, 64))
    assert torch.equal(sf[:, 0, 0].view(g // 1000, 1000), words[:, :1000].expand(g // 1000, 1000))
    y = fp8bs.dequantize_mxfp4(q, sf)
    assert torch.equal(y.view(g // 1000, 1000, 128),
                       fp8bs.dequantize_mxfp4(want, words).expand(g // 1000, 1000, 128))


@pytest.mark.parametrize("g,max_m,n,k", SLOTS + [(16, 256, 4096, 7168)])
@pytest.mark.parametrize("most", [1, 16, 17, 32, 33, 64, 65, 128, 129])
def test_the_hint_changes_no_result_of_slots_with_few_rows(gen, g, max_m, n, k, most):
    # counts up to limits at which other kernels may take the slots, and one past them
    if most > max_m:
        pytest.skip("more rows than a slot has")
    a, sfa = operand(gen, g, max_m, k)
    b, sfb = operand(gen, g, n, k)
    masked = torch.tensor([(37 * i + 11) % (most + 1) for i in range(g)], dtype=torch.int32, device="cuda")
    masked[0] = most
    runs = []
    for expected in (0, 1, 40, max_m):
        d = torch.zeros(g, max_m, n, dtype=torch.bfloat16, device="cuda")
        fp8bs.fp8bs_grouped_masked_nt_mxfp4(a, sfa, b, sfb, d, masked, expected_m=expected)
        runs.append(d)
    assert all(torch.equal(d, runs[0]) for d in runs[1:])
    assert runs[0][0, :most].any(-1).all() and not runs[0][0, most:].any()
    rows = torch.arange(max_m, device="cuda")[None] < masked[:, None]
    assert torch.equal(runs[0].any(-1), rows)
