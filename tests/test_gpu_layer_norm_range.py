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
