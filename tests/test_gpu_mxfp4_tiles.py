"""GPU tests of the MXFP4 operators' kernels one by one against their definitions in 64 bits,
with the bounds that tests/test_gpu_mxfp4.py derives."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs
from test_gpu_mxfp4 import _act, _say, backward_bounds, bf16, matrix, near, pack, values

pytestmark = pytest.mark.gpu


# ---- gates of any size ---------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m", [3, 1200])
def test_gradients_at_gates_whose_powers_overflow(m, act):
    # the gate is +-2^p, the up projection 0.5: both gradients are finite for every p here, though
    # the square and the cube of the gate need not be (32-bit numbers end at 2^128)
    _say(f"[gpu] gates 2^p, {m} rows, {act}")
    f, k = 32, 128
    power = np.array([-60, -3, 0, 2, 4, 10, 20, 42, 43, 50, 63, 64, 70, 80, 90, 100])
    ca, ea = np.zeros((m, k), np.uint8), np.full((m, k // 32), 127, np.uint8)
    ca[:, 0] = ca[:, 32] = 2                              # 1.0, for the gate and for up
    cb, eb = np.zeros((2 * f, k), np.uint8), np.full((2 * f, k // 32), 127, np.uint8)
    cb[:f, 0] = np.where(np.arange(f) % 2, 10, 2)         # -1.0, 1.0
    eb[:f, 0] = 127 + power[np.arange(f) // 2]
    cb[f:, 32] = 1                                        # 0.5
    a, b = values(ca, ea), values(cb, eb)
    dh = bf16(np.random.default_rng(m).choice([-1.5, 0.25, 1.0], (m, f)))
    d64 = dh.double().numpy()
    gate, up = a @ b[:f].T, a @ b[f:].T
    v, slope = _act(gate, act)
    da = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    db = torch.empty(2 * f, k, device="cuda")
    fp8bs.fp8bs_gated_dense_mxfp4_backward(*pack(ca, ea), *pack(cb, eb), dh.cuda(), da, db, activation=act)
    dg, du = d64 * up * slope, d64 * v
    # Sums of terms of every size in one row or column: bounded by the terms' own rounding to
    # bf16, 2^-8, and by the activation's error of 40 units in the last place of |gate| at most
    # (the exponential's argument is rounded, but is 0 beyond |gate| = 100), and the output's.
    rel = 2.0 ** -8 + 2.0 ** -12
    size = np.abs(np.concatenate((dg, du), 1))
    want_a = np.concatenate((dg, du), 1) @ b
    want_b = np.concatenate((dg, du), 1).T @ a
    tiny = 2.0 ** -100
    near(da, want_a, 2.2 * rel * (size @ np.abs(b)) + tiny, "da")
    near(db, want_b, 2.2 * rel * (size.T @ np.abs(a)) + tiny, "db")
