"""The norm and its gradients at the ends of FP32's range (`-m gpu`), against their definitions in 64
bits; bounds as in tests/test_gpu_layer_norm.py."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs
from _layer_ref import E, host

pytestmark = pytest.mark.gpu
F32 = torch.float32

# one, four and sixteen wavefronts a row, one to four eights a lane
SHAPES = [(5, 256), (5, 1000), (600, 1000), (600, 2048), (5, 7168), (600, 7168), (5, 16384), (5, 32768)]


def norm(x, w, eps):
    y, rstd = torch.empty_like(x), torch.empty(len(x), device="cuda")
    fp8bs.fp8bs_rms_norm(x, w, y=y, rstd=rstd, eps=eps)
    s = host(x).astype(np.float64)
    want = 1 / np.sqrt((s * s).mean(-1) + float(np.float32(eps)))
    return host(y), host(rstd), s * want[:, None] * host(w).astype(np.float64), want


def check(x, w, eps):
    y, rstd, want_y, want = norm(x, w, eps)
    # (a reciprocal below 2^-126 keeps fewer bits, a value below it too)
    assert np.all(np.abs(rstd - want) <= 34 * E * want + 2.0 ** -149)
    assert np.all(np.abs(y - want_y) <= 40 * E * np.abs(want_y) + 1e-38)


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("eps", [1e-6, 1e34, 1e36, 2e38, 3e38])
def test_squares_that_overflow_with_their_eps(rows, k, eps):
    """the sum of squares overflows, or only their mean with eps: eps counts all the same"""
    gen = torch.Generator("cuda").manual_seed(k)
    x = torch.rand(rows, k, generator=gen, device="cuda") - 0.5
    x *= torch.tensor([1e10, 1e18, 3e19, 1e25, 3e38], device="cuda").repeat(rows // 5)[:, None]
    check(x, 1 + torch.rand(k, generator=gen, device="cuda"), eps)


# lanes past the last column read the last weights again
@pytest.mark.parametrize("rows,k", [(3, 8), (3, 264), (1100, 264), (3, 1000), (500, 1000), (3, 3000), (400, 3000),
                                    (3, 7000), (600, 7000), (1100, 7000), (3, 9000), (3, 20000)])
@pytest.mark.parametrize("place", [0, -1])
def test_gradients_of_an_infinite_weight(rows, k, place):
    gen = torch.Generator("cuda").manual_seed(k)
    s, dy, dres = (torch.randn(rows, k, generator=gen, device="cuda") for _ in range(3))
    rstd, w = 1 / torch.sqrt(s.square().mean(-1)), 1 + torch.rand(k, generator=gen, device="cuda")
    w[place] = float("inf")
    dx, dw = torch.empty_like(s), torch.empty(k, device="cuda")
    fp8bs.fp8bs_rms_norm_backward(s, rstd, w, dy, dx, dres, dw)
    s, r, w, dy, dres = (host(t).astype(np.float64) for t in (s, rstd, w, dy, dres))
    h, g = s * r[:, None], dy * w
    with np.errstate(invalid="ignore"):
        want = dres + r[:, None] * (g - h * (g * h).mean(-1, keepdims=True))
    # an infinite mean makes all of a row infinite but the weight's own column, a difference of infinities
    assert np.isinf(np.delete(want, place % k, 1)).all() and np.isnan(want[:, place]).all()
    assert np.array_equal(host(dx), want, equal_nan=True)
    assert np.isfinite(host(dw)).all()


@pytest.mark.parametrize("rows,k", SHAPES)
def test_small_values_beside_squares_that_overflow(rows, k):
    gen = torch.Generator("cuda").manual_seed(k)
    x = torch.rand(rows, k, generator=gen, device="cuda") - 0.5
    x[:, 0] = 4e19                                 # (its square alone overflows)
    x[:, 1:] *= torch.logspace(-17, 15, k - 1, device="cuda")
    check(x, 1 + torch.rand(k, generator=gen, device="cuda"), 1e-6)


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("eps", [1e-6, 2.0 ** -120, 2.0 ** -126, 1e-40, 1e-43, 2.0 ** -149])
def test_squares_and_eps_below_the_normal_range(rows, k, eps):
    """mean and eps that are no normal numbers: statistics to FP32's precision all the same"""
    gen = torch.Generator("cuda").manual_seed(k)
    x = torch.rand(rows, k, generator=gen, device="cuda") - 0.5
    x *= torch.tensor([0.0, 1e-18, 3e-20, 1e-21, 1e-23], device="cuda").repeat(rows // 5)[:, None]
    check(x, 1 + torch.rand(k, generator=gen, device="cuda"), eps)
