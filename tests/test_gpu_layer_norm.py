"""GPU tests of the root-mean-square norm with residual and e4m3 output, and of its gradients,
against their definitions in 64 bits.

Bounds (E = 2^-24 an FP32 rounding).  The sum of k squares is added in chains of at most 32 terms
of a lane, then 6 exchanges and up to 16 wavefronts: 56 roundings of positive terms at most, so
mean s^2 is off by 58 E relative, 1 / sqrt(...) by half of that and 3 roundings, y by two products
and the sum s = x + residual more: 40 E relative, and E |s| rstd |w| where s is a sum.  The mean of
g h in the backward pass is off by 62 E times the mean of |g h|; dweight, over rows, by one rounding
for each row of a part (at most rows / 512 + 4), 2 where four rows' sums are joined, 48 for the sum of
up to 512 parts in 32 chains and 3 of each term."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs
import _layer_ref as ref
from _layer_ref import E, HALF, host

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rand(gen, *shape, dtype=BF16, size=1.0):
    x = torch.randn(shape, generator=gen, device="cuda") * size
    return (x * torch.exp(0.5 * torch.randn(shape[0], *[1] * (len(shape) - 1), generator=gen,
                                            device="cuda"))).to(dtype)


@pytest.fixture
def gen():
    return torch.Generator("cuda").manual_seed(11)


def expected(x, w, res, eps):
    s = host(x).astype(np.float64) + (0 if res is None else host(res).astype(np.float64))
    rstd = 1 / np.sqrt((s * s).mean(-1) + eps)
    w = host(w).astype(np.float64)
    with np.errstate(invalid="ignore"):
        y = s * rstd[:, None] * w
    added = 0 if res is None else E * (np.abs(s) + 1e-38) * rstd[:, None] * np.abs(w)
    return s, rstd, y, 40 * E * np.abs(y) + added + 1e-38


# every kernel: few rows (fewer than 512) on as many wavefronts as a row fills, many rows; 1, 2 and 4
# eights a lane of 1, 4 and 16 wavefronts; rows that are no multiple of a workgroup's four
SHAPES = [(1, 128), (3, 384), (1, 2048), (63, 640), (65, 1920), (2, 7168), (5, 8192), (2, 9088),
          (3, 16384), (1, 17024), (2, 32768), (512, 128), (515, 512), (514, 640), (513, 1024),
          (517, 2048), (512, 2176), (515, 4096), (513, 4224), (520, 7168), (512, 8320), (513, 16512)]


@pytest.mark.parametrize("rows,k", SHAPES)
def test_norm_with_residual_and_codes(gen, rows, k):
    print(f"[gpu] norm {rows}x{k}", flush=True)
    x, res = rand(gen, rows, k), rand(gen, rows, k)
    w = (1 + 0.2 * torch.randn(k, generator=gen, device="cuda")).to(BF16)
    out, y = torch.empty_like(res), torch.empty(rows, k, device="cuda")
    q = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    sfa = torch.full((k // 128, fp8bs.get_sfa_ld(rows)), -7.0, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    fp8bs.fp8bs_rms_norm(x, w, res, out, y, q, sfa, rstd, eps=1e-5)
    s, want_rstd, want, tol = expected(x, w, res, 1e-5)
    assert np.all(np.abs(host(rstd) - want_rstd) <= 34 * E * want_rstd)
    assert np.array_equal(host(out), ref.bf16(host(x) + host(res)))
    assert np.all(np.abs(host(y) - want) <= tol)
    # the codes are those of y's FP32 values, bit for bit
    code, scale = ref.quantise(host(y), -1)
    assert np.array_equal(host(q), code)
    assert np.array_equal(ref.row_scales(sfa, rows), scale)
    assert np.all(host(sfa)[:, rows:] == -7.0)
    # y in bf16 is the same value rounded once, and the outputs do not depend on each other
    y16, q2, sfa2 = torch.empty_like(x), torch.zeros_like(q), torch.zeros_like(sfa)
    fp8bs.fp8bs_rms_norm(x, w, res, y=y16, eps=1e-5)
    assert torch.equal(y16, y.to(BF16))
    fp8bs.fp8bs_rms_norm(x, w, res, q=q2, sfa=sfa2, eps=1e-5)
    assert torch.equal(q2, q) and torch.equal(sfa2[:, :rows], sfa[:, :rows])


@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("rows,k", [(7, 1000), (530, 264), (530, 3000)])
def test_norm_types_and_sizes_of_eights(gen, xt, rt, wt, rows, k):
    x = rand(gen, rows, k, dtype=xt)
    res = None if rt is None else rand(gen, rows, k, dtype=rt)
    w = (1 + 0.2 * torch.randn(k, generator=gen, device="cuda")).to(wt)
    y, rstd = torch.empty(rows, k, device="cuda"), torch.empty(rows, device="cuda")
    out = torch.empty(rows, k, dtype=rt or BF16, device="cuda")
    fp8bs.fp8bs_rms_norm(x, w, res, out, y, rstd=rstd)
    s, want_rstd, want, tol = expected(x, w, res, 1e-6)
    assert np.all(np.abs(host(y) - want) <= tol)
    summed = host(x) if res is None else host(x) + host(res)
    assert np.array_equal(host(out), ref.bf16(summed) if out.dtype == BF16 else summed)
    assert np.all(np.abs(host(rstd) - want_rstd) <= 34 * E * want_rstd)


def test_norm_in_place_and_allocating(gen):
    x, res = rand(gen, 33, 1280), rand(gen, 33, 1280)
    w = (1 + 0.2 * torch.randn(1280, generator=gen, device="cuda")).to(BF16)
    y, out = torch.empty_like(x), torch.empty_like(x)
    fp8bs.fp8bs_rms_norm(x, w, res, out, y)
    q, sfa, s, rstd = fp8bs.rms_norm_1x128(x, w, res)
    fp8bs.fp8bs_rms_norm(x, w, res, residual_out=res, y=x)
    assert torch.equal(x, y) and torch.equal(res, out) and torch.equal(s, out)
    code, scale = ref.quantise(host(y), -1)        # (of bf16 values: near, not the same)
    got = ref.values_1x128(q, sfa)
    assert np.linalg.norm(got - host(y)) < 2.0 ** -4 * np.linalg.norm(host(y))
    q2, _, s2, _ = fp8bs.rms_norm_1x128(s, w)
    assert s2 is s


def test_norm_rows_at_the_ends_of_the_range():
    k = 1024
    x = torch.zeros(9, k, device="cuda")
    x[1] = 1e-30                               # far below eps
    x[2] = 1e25                                # the squares overflow
    x[3, :500] = 3e38
    x[4] = torch.linspace(-3e19, 3e19, k, device="cuda")
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x[7] = 1e18                                # the sum of squares overflows, not their mean
    x[8] = 1.0
    w = torch.full((k,), 0.5, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(9, device="cuda")
    q, sfa = torch.zeros(9, k, dtype=torch.uint8, device="cuda"), torch.zeros(8, 12, device="cuda")
    fp8bs.fp8bs_rms_norm(x, w, y=y, q=q, sfa=sfa, rstd=rstd, eps=1e-6)
    s, want_rstd, want, tol = expected(x, w, None, 1e-6)
    fine = [0, 1, 2, 3, 4, 7, 8]
    assert np.all(np.abs(host(y) - want)[fine] <= tol[fine])
    # (a reciprocal below 2^-126 keeps fewer bits)
    assert np.all(np.abs(host(rstd) - want_rstd)[fine] <= (34 * E * want_rstd + 2.0 ** -149)[fine])
    assert host(rstd)[5] == 0 and np.isnan(host(y)[5, 7]) and np.all(np.delete(host(y)[5], 7) == 0)
    assert np.isnan(host(y)[6]).all()
    code, scale = ref.quantise(host(y), -1)
    assert ref.same_codes(host(q), code) and np.array_equal(ref.row_scales(sfa, 9), scale)
    assert np.all(host(q)[0] == 0) and np.all(host(q)[6] & 127 == 127)


def gradients(s, rstd, w, dy, dres):
    s, r, w, dy = (host(t).astype(np.float64) for t in (s, rstd, w, dy))
    h, g = s * r[:, None], dy * w
    mean = (g * h).mean(-1, keepdims=True)
    dres = 0 if dres is None else host(dres).astype(np.float64)
    dx = dres + r[:, None] * (g - h * mean)
    off = r[:, None] * (6 * E * np.abs(g) + np.abs(h) * (
        6 * E * np.abs(mean) + 62 * E * np.abs(g * h).mean(-1, keepdims=True)))
    return dx, off + 2 * E * np.abs(dx) + 2 * E * np.abs(dres) + 1e-38, (dy * h).sum(0), np.abs(dy * h).sum(0)


@pytest.mark.parametrize("rows,k", [(1, 128), (1, 8), (3, 1000), (300, 512), (200, 2048), (64, 7168),
                                    (2, 9000), (1, 32768), (512, 504), (2060, 512), (700, 1024),
                                    (515, 2048), (600, 4096), (1030, 7168), (1024, 4608), (513, 16384),
                                    (512, 20000), (384, 16384), (385, 2048), (384, 4096)])
@pytest.mark.parametrize("st,gt,wt", [(BF16, BF16, BF16), (F32, BF16, F32), (BF16, F32, F32),
                                      (F32, F32, BF16)])
def test_gradients(gen, rows, k, st, gt, wt):
    print(f"[gpu] norm gradients {rows}x{k} {st} {gt} {wt}", flush=True)
    s, dy = rand(gen, rows, k, dtype=st), rand(gen, rows, k, dtype=gt, size=0.1)
    dres = rand(gen, rows, k, dtype=st, size=0.1)
    w = (1 + 0.2 * torch.randn(k, generator=gen, device="cuda")).to(wt)
    rstd = 1 / torch.sqrt(s.float().square().mean(-1) + 1e-6)
    dx, dw = torch.empty_like(s), torch.full((k,), 3.0, device="cuda")
    fp8bs.fp8bs_rms_norm_backward(s, rstd, w, dy, dx, dres, dw)
    want, tol, want_w, size_w = gradients(s, rstd, w, dy, dres)
    assert np.all(np.abs(host(dx) - want) <= tol + HALF[st] * (np.abs(want) + tol))
    tol_w = (rows / 512 + 4 + 2 + 48 + 3) * E * size_w + 1e-38
    assert np.all(np.abs(host(dw) - want_w) <= tol_w)
    # added to what is there; without the residual's gradient, without dweight
    more = torch.full((k,), 3.0, device="cuda")
    fp8bs.fp8bs_rms_norm_backward(s, rstd, w, dy, dx, None, more, accumulate=True)
    assert torch.equal(more, dw + 3.0)
    want, tol, _, _ = gradients(s, rstd, w, dy, None)
    assert np.all(np.abs(host(dx) - want) <= tol + HALF[st] * (np.abs(want) + tol))
    other = torch.empty_like(s)
    fp8bs.fp8bs_rms_norm_backward(s, rstd, w, dy, other)
    assert torch.equal(other, dx)


def test_gradients_are_the_formulas(gen):
    """the reference's gradients against differences and autograd in 64 bits"""
    rng = np.random.default_rng(3)
    x, w, dy, dres = rng.normal(size=(4, 24)), rng.normal(size=24), rng.normal(size=(4, 24)), rng.normal(size=(4, 24))
    eps = 1e-3
    t = [torch.from_numpy(v).requires_grad_() for v in (x, w)]
    y = t[0] / torch.sqrt((t[0] ** 2).mean(-1, keepdim=True) + eps) * t[1]
    (y * torch.from_numpy(dy)).sum().backward()
    rstd = 1 / np.sqrt((x * x).mean(-1) + eps)
    as_t = lambda v: torch.from_numpy(v)  # noqa: E731
    dx, _, dw, _ = gradients(as_t(x), as_t(rstd), as_t(w), as_t(dy), as_t(dres))
    assert np.allclose(dx, t[0].grad.numpy() + dres, rtol=1e-12, atol=1e-12)
    assert np.allclose(dw, t[1].grad.numpy(), rtol=1e-12)

    def loss(x):
        return (x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w * dy).sum() + (x * dres).sum()
    d = rng.normal(size=x.shape)
    numeric = (loss(x + 1e-5 * d) - loss(x - 1e-5 * d)) / 2e-5
    assert abs(numeric - (dx * d).sum()) < 1e-7 * np.abs(dx * d).sum()


@pytest.mark.parametrize("rows,k", [(1, 128), (70, 896), (384, 264), (385, 264), (384, 1000), (200, 7168), (384, 16384),
                                    (600, 7168)])
def test_gradients_in_place_with_dweight(gen, rows, k):
    """few rows' dweight is added from the inputs: the same whether dx is written over them or not"""
    s, dy, dres = rand(gen, rows, k), rand(gen, rows, k), rand(gen, rows, k)
    w = (1 + 0.2 * torch.randn(k, generator=gen, device="cuda"))
    rstd = 1 / torch.sqrt(s.float().square().mean(-1) + 1e-6)
    dx, dw = torch.empty_like(s), torch.empty(k, device="cuda")
    fp8bs.fp8bs_rms_norm_backward(s, rstd, w, dy, dx, dres, dw)
    _, _, want_w, size_w = gradients(s, rstd, w, dy, dres)
    # (chains of every 32nd or 128th row at least, their sums by halves, three roundings of a product)
    assert np.all(np.abs(host(dw) - want_w) <= (rows / 32 + 1 + 7 + 3) * E * size_w + 1e-38)
    for i in range(3):
        for _ in range(5):
            args, own = [s.clone(), dy.clone(), dres.clone()], torch.empty(k, device="cuda")
            fp8bs.fp8bs_rms_norm_backward(args[0], rstd, w, args[1], args[i], args[2], own)
            assert torch.equal(args[i], dx) and torch.equal(own, dw)


def test_gradients_in_place_and_of_no_rows(gen):
    s, dy, dres = rand(gen, 70, 896), rand(gen, 70, 896), rand(gen, 70, 896)
    w = (1 + 0.2 * torch.randn(896, generator=gen, device="cuda"))
    rstd = 1 / torch.sqrt(s.float().square().mean(-1) + 1e-6)
    want = torch.empty_like(s)
    fp8bs.fp8bs_rms_norm_backward(s, rstd, w, dy, want, dres)
    for i in range(3):
        args = [s.clone(), dy.clone(), dres.clone()]
        fp8bs.fp8bs_rms_norm_backward(args[0], rstd, w, args[1], args[i], args[2])
        assert torch.equal(args[i], want)
    empty = torch.empty(0, 896, dtype=BF16, device="cuda")
    dw = torch.full((896,), 5.0, device="cuda")
    none = torch.empty(0, device="cuda")
    fp8bs.fp8bs_rms_norm_backward(empty, none, w, empty, empty.clone(), None, dw, accumulate=True)
    assert bool((dw == 5.0).all())
    fp8bs.fp8bs_rms_norm_backward(empty, none, w, empty, empty.clone(), None, dw)
    assert bool((dw == 0.0).all())
    fp8bs.fp8bs_rms_norm(empty, w, y=empty.clone())


def test_the_cap_changes_no_result(gen):
    for rows in (3000, 300):
        caps_agree(rand(gen, rows, 640), rand(gen, rows, 640), gen)


def caps_agree(s, dy, gen):
    w = (1 + 0.2 * torch.randn(640, generator=gen, device="cuda"))
    runs = []
    try:
        for cap in (0, 3, 40):
            fp8bs.set_num_cus(cap)
            q, sfa, _, rstd = fp8bs.rms_norm_1x128(s, w)
            dx, dw = torch.empty_like(s), torch.empty(640, device="cuda")
            fp8bs.fp8bs_rms_norm_backward(s, rstd, w, dy, dx, None, dw)
            runs.append((q, sfa, rstd, dx, dw))
    finally:
        fp8bs.set_num_cus(0)
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_rows_past_4_gib(gen):
    rows, k = 330000, 8192
    x = torch.zeros(rows, k, dtype=BF16, device="cuda")
    last = rand(gen, 5, k)
    x[-5:] = last
    w = torch.ones(k, device="cuda", dtype=BF16)
    q, sfa, _, rstd = fp8bs.rms_norm_1x128(x, w)
    # (rows enough for the same layout over wavefronts, so the same order of sums)
    q1, sfa1, _, rstd1 = fp8bs.rms_norm_1x128(torch.cat([x[:1100], last]), w)
    assert torch.equal(q[-5:], q1[-5:]) and torch.equal(rstd[-5:], rstd1[-5:])
    assert torch.equal(sfa[:, rows - 5:rows], sfa1[:, 1100:1105])
    dx = torch.empty_like(x)
    fp8bs.fp8bs_rms_norm_backward(x, rstd, w, x, dx)
    dx1 = torch.empty(1105, k, dtype=BF16, device="cuda")
    fp8bs.fp8bs_rms_norm_backward(torch.cat([x[:1100], last]), rstd1, w, torch.cat([x[:1100], last]), dx1)
    assert torch.equal(dx[-5:], dx1[-5:])


def test_refusals_on_the_device(gen):
    x, w = rand(gen, 4, 256), torch.ones(256, device="cuda")
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.fp8bs_rms_norm(rand(gen, 4, 252), torch.ones(252, device="cuda"), y=torch.empty(4, 252, device="cuda"))
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.fp8bs_rms_norm(x, w, y=x, eps=0.0)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_rms_norm(x, w)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_rms_norm(x, w[:128], y=x)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_rms_norm(x.t(), w, y=x)
    with pytest.raises(TypeError):
        fp8bs.fp8bs_rms_norm(x.half(), w, y=x)
    with pytest.raises(TypeError):
        fp8bs.fp8bs_rms_norm(x, w, x, x.float())
    with pytest.raises(ValueError):
        fp8bs.fp8bs_rms_norm(x, w, q=torch.empty(4, 256, dtype=torch.uint8, device="cuda"))
    rstd = torch.ones(4, device="cuda")
    with pytest.raises(TypeError):
        fp8bs.fp8bs_rms_norm_backward(x, rstd, w, x, x.float())
    with pytest.raises(ValueError):
        fp8bs.fp8bs_rms_norm_backward(x, rstd[:3], w, x, x)
    x, rstd = rand(gen, 400, 256), torch.ones(400, device="cuda")
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.fp8bs_rms_norm_backward(x, rstd, w, x, x, None, w.clone(),
                                      workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
