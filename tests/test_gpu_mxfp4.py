"""GPU tests of the MXFP4 operators against their definitions in 64 bits (numpy): the
quantiser and its inverse bit for bit, products, the gated block, its backward pass and the
feed-forward layer within bounds derived from the roundings they make.

Bounds.  half(x) = 2^(floor(log2 |x|) - 8) is half a bf16 unit in the last place (8
significant bits), at most u |x| with u = 2^-8; e = 2^-24 bounds an FP32 rounding.  A product
sums k terms in FP32: error <= (k + 8) e * S with S = sum |a_i b_i| (any order; the 8 covers
the matrix core's alignment of a 128-term block).  Then one rounding to bf16.  Activations use v_exp_f32 and
v_rcp_f32 (each within 2 FP32 units here bounded by 16 e relative, on inputs of moderate
size: exp's argument reduction adds |v| e).
"""
import itertools
import sys

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
U, E = 2.0 ** -8, 2.0 ** -24


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


# ---- definitions in 64 bits ----------------------------------------------------

def quantise(x):
    """codes [.., k] and exponents [.., k/32] of float values, from the definition"""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.max(np.abs(b), axis=-1)
    bad = ~np.isfinite(b).all(axis=-1)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    e = np.floor(np.log2(safe)).astype(np.int64)
    e = np.where(2.0 ** (e + 1) <= safe, e + 1, np.where(2.0 ** e > safe, e - 1, e))
    e = np.where(amax == 0, -10 ** 6, e)
    e = np.maximum(e - 2, -127)
    with np.errstate(invalid="ignore"):
        v = np.where(bad[..., None], 0.0, b) * 2.0 ** (-e[..., None].astype(np.float64))
    mag = np.abs(v)
    grid = E2M1[:8]
    d = np.abs(mag[..., None] - grid)
    best = d.min(-1, keepdims=True)
    # nearest; of two equally near the even code
    near = d == best
    pick = np.where(near, np.arange(8) % 2 * 16 + np.arange(8), 99).argmin(-1)
    code = pick + 8 * np.signbit(v)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values(code, e):
    v = E2M1[code].reshape(*code.shape[:-1], -1, 32)
    s = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(code.shape)


def pack(code, e, pad=0):
    """device tensors (codes, exponents) in the operators' layout"""
    q = (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)
    rows, kb = e.shape[-2], e.shape[-1]
    ld = fp8bs.get_sfa_ld(rows)
    sf = np.full(e.shape[:-2] + (kb // 4, ld, 4), pad, dtype=np.uint8)
    sf[..., :rows, :] = np.moveaxis(e.reshape(*e.shape[:-1], kb // 4, 4), -3, -2)
    return (torch.from_numpy(q).cuda(),
            torch.from_numpy(np.ascontiguousarray(sf).view(np.int32)[..., 0].copy()).cuda())


def unpack(q, sf, rows):
    q, sf = q.cpu().numpy(), sf.cpu().numpy()
    code = np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)
    b = np.ascontiguousarray(sf)[..., None].view(np.uint8)
    pad = b[..., rows:, :]
    e = np.moveaxis(b[..., :rows, :], -3, -2)
    return code, e.reshape(*e.shape[:-2], 4 * e.shape[-2]), pad


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def _act(v, name):
    if name == "silu":
        s = 1 / (1 + np.exp(-v))
        return v * s, s * (1 + v * (1 - s))
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 0.134145 * v * v)


def matrix(rng, shape, scale=1.0, spread=0.5):
    """random codes and exponents, packed, and the values they stand for"""
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,))) * scale
    code, e = quantise(x)
    return code, e, values(code, e)


def half(x):
    """half a bf16 unit in the last place"""
    x = np.abs(x)
    return 2.0 ** (np.floor(np.log2(np.where(x > 0, x, 1.0))) - 8) * (x > 0)


def rounded(want, err):
    """bound on the bf16 rounding of a value within err of want"""
    return err + half(np.abs(want) + err)


def near(got, want, bound, what):
    got = got.detach().cpu().double().numpy()
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} out of bounds, first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]} vs {want[bad][0]}")


def product_bound(x, w):
    """(|error| of the FP32 sum, value)"""
    k = x.shape[-1]
    return (k + 8) * E * (np.abs(x) @ np.abs(w).T), x @ w.T


def gated_bound(x, w, f, act):
    """value of h, and a bound on the error of its FP32 form"""
    eg, g = product_bound(x, w[:f])
    eu, u = product_bound(x, w[f:])
    v, slope = _act(g, act)
    # |act'| <= 1.13 for both; the activation's own arithmetic
    ea = 1.13 * eg + (16 + np.abs(g)) * E * np.maximum(np.abs(v), np.abs(g) * 2.0 ** -20)
    return v * u, ea * np.abs(u) + np.abs(v) * eu + 2 * ea * eu + 4 * E * np.abs(v * u)


SENTINEL = 77.0


# ---- quantiser -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 128), (31, 256), (33, 384), (64, 1152), (3, 70, 256),
                                   (300, 2048)])
def test_quantiser_and_inverse(shape, dtype):
    _say(f"[gpu] quantize_mxfp4 {shape} {dtype}")
    rng = np.random.default_rng(sum(shape))
    x = rng.standard_normal(shape).astype(np.float32)
    x *= np.exp2(rng.integers(-30, 30, shape[:-1] + (shape[-1] // 32,))).repeat(32, -1)
    flat = x.reshape(-1, 32)
    flat[0] = 0
    flat[1] = -0.0
    t = torch.from_numpy(x).to(dtype)
    x = t.double().numpy()
    k, rows = shape[-1], shape[-2]
    q = torch.full(shape[:-1] + (k // 2,), 0xAB, dtype=torch.uint8, device="cuda")
    sf = torch.full(shape[:-2] + (k // 128, fp8bs.get_sfa_ld(rows)), 0x5A5A5A5A,
                    dtype=torch.int32, device="cuda")
    fp8bs.fp8bs_quantize_mxfp4(t.cuda(), q, sf)
    code, e, pad = unpack(q, sf, rows)
    want, want_e = quantise(x)
    assert np.array_equal(e, want_e)
    assert np.array_equal(code, want)
    assert (pad == 0x5A).all()
    for out in (torch.bfloat16, torch.float32):
        y = fp8bs.dequantize_mxfp4(q, sf, out)
        assert y.dtype == out
        assert np.array_equal(y.cpu().double().numpy(), values(want, want_e))


def test_quantiser_ties_saturation_and_exponents():
    # every tie between neighbouring codes and the floats next to it, both signs, at the
    # smallest, a middle and the largest exponents
    mids = (E2M1[:7] + E2M1[1:8]) / 2
    pts = np.concatenate([mids, [5.0, 6.5, 7.0, 7.9999995, 0.0, 0.25]]).astype(np.float32)
    pts = np.concatenate([pts, np.nextafter(pts, np.float32(0)), np.nextafter(pts, np.float32(9))])
    pts = pts[pts < 8]
    rows = []
    for scale in (-127, -126, -100, -1, 0, 1, 90, 125):
        for sign in (1, -1):
            v = np.zeros((pts.size + 30) // 31 * 32, np.float64)
            i = np.arange(pts.size)
            v[i // 31 * 32 + i % 31] = pts * sign
            v[31::32] = 4.0                               # fixes the block's exponent
            rows.append(np.pad(v, (0, -v.size % 128)) * 2.0 ** scale)
    x = np.array(rows).astype(np.float32)
    q, sf = fp8bs.quantize_mxfp4(torch.from_numpy(x).cuda())
    code, e, _ = unpack(q, sf, x.shape[0])
    want, want_e = quantise(x.astype(np.float64))
    assert np.array_equal(e, want_e)
    assert np.array_equal(code, want)


def test_quantiser_of_every_bf16_value():
    # each finite bf16 value twice: with nothing larger in its block, and two octaves below
    # its block's largest
    bits = np.arange(65536, dtype=np.uint32)
    x = (bits << 16).view(np.float32)
    x = x[np.isfinite(x)]
    own = np.zeros((x.size, 32), np.float32)
    own[:, 5] = x
    beside = own.copy()
    with np.errstate(over="ignore"):
        big = x * np.float32(4)
    beside[:, 9] = np.where(np.isfinite(big), big, 0)
    v = np.concatenate([own, beside])
    v = np.pad(v, ((0, -len(v) % 8), (0, 0))).reshape(-1, 256)
    t = torch.from_numpy(v).bfloat16()
    assert np.array_equal(t.float().numpy(), v)
    want, want_e = quantise(v.astype(np.float64))
    for inp in (t, torch.from_numpy(v)):
        q, sf = fp8bs.quantize_mxfp4(inp.cuda())
        code, e, _ = unpack(q, sf, len(v))
        assert np.array_equal(e, want_e)
        assert np.array_equal(code, want)


def test_quantiser_infinities_nans_and_subnormals():
    x = np.random.default_rng(5).standard_normal((6, 256)).astype(np.float32)
    x[0, 3] = np.inf
    x[1, 40] = -np.inf
    x[2, 100] = np.nan
    x[3, 128:160] = np.float32(1e-42)                     # subnormal block
    x[4, 32:64] = 2.0 ** -124
    x[5, 64:96] = np.finfo(np.float32).max
    q, sf = fp8bs.quantize_mxfp4(torch.from_numpy(x).cuda())
    code, e, _ = unpack(q, sf, 6)
    want, want_e = quantise(x.astype(np.float64))
    assert np.array_equal(e, want_e)
    assert np.array_equal(code, want)
    assert e[0, 0] == e[1, 1] == e[2, 3] == 255
    y = fp8bs.dequantize_mxfp4(q, sf, torch.float32).cpu().double().numpy()
    v = values(want, want_e)
    assert np.array_equal(y, v, equal_nan=True) and np.isnan(y[0, :32]).all()


def test_inverse_of_every_code_and_exponent():
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 8))          # [256][128]
    e = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, 1)
    q, sf = pack(code, e)
    v = values(code, e)
    with np.errstate(over="ignore"):
        f32 = v.astype(np.float32)
    y = fp8bs.dequantize_mxfp4(q, sf, torch.float32).cpu().numpy()
    assert np.array_equal(y, f32, equal_nan=True)
    y = fp8bs.dequantize_mxfp4(q, sf).cpu()
    assert np.array_equal(y.float().numpy(), torch.from_numpy(f32).bfloat16().float().numpy(),
                          equal_nan=True)


# ---- products ------------------------------------------------------------------

DENSE = [(1, 1, 128), (1, 300, 384), (3, 129, 128), (16, 64, 256), (17, 65, 640), (64, 256, 1024),
         (65, 1000, 512), (128, 2112, 896), (200, 130, 256), (333, 515, 1152), (600, 700, 384),
         (2100, 2049, 256)]


@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense_product(m, n, k):
    _say(f"[gpu] dense_nt_mxfp4 {m} {n} {k}")
    rng = np.random.default_rng(m + n + k)
    ca, ea, a = matrix(rng, (m, k))
    cb, eb, b = matrix(rng, (n, k))
    d = torch.full((m + 1, n), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_dense_nt_mxfp4(*pack(ca, ea, 255), *pack(cb, eb, 255), d[:m])
    err, want = product_bound(a, b)
    near(d[:m], want, rounded(want, err), f"dense {m}x{n}x{k}")
    assert (d[m] == SENTINEL).all()


def test_product_takes_the_scales_of_every_block():
    # one value per block is not zero: each result is one product of two scales
    m, n, k = 20, 40, 512
    rng = np.random.default_rng(9)
    code = np.zeros((m, k), np.uint8)
    code[:, ::32] = 2                                      # 1.0
    ea = rng.integers(100, 150, (m, k // 32)).astype(np.uint8)
    cb = np.zeros((n, k), np.uint8)
    block = np.arange(n) % (k // 32)
    cb[np.arange(n), 32 * block] = 2
    eb = rng.integers(100, 150, (n, k // 32)).astype(np.uint8)
    d = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_dense_nt_mxfp4(*pack(code, ea), *pack(cb, eb), d)
    want = values(code, ea) @ values(cb, eb).T
    assert np.array_equal(d.cpu().double().numpy(), want)


def test_nan_scales_stay_in_their_rows_and_columns():
    m, n, k = 70, 90, 384
    rng = np.random.default_rng(3)
    ca, ea, a = matrix(rng, (m, k))
    cb, eb, b = matrix(rng, (n, k))
    ea[5, 11] = 255
    eb[33, 0] = 255
    d = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_dense_nt_mxfp4(*pack(ca, ea), *pack(cb, eb), d)
    got = np.isnan(d.cpu().float().numpy())
    want = np.zeros((m, n), bool)
    want[5] = want[:, 33] = True
    assert np.array_equal(got, want)


def contiguous_layout(rng, blocks_of, pads):
    """(grouped_layout, [(start, end, expert)]) from (expert, blocks) runs"""
    total = 128 * sum(n for _, n in blocks_of)
    index = np.full(total, -1, np.int32)
    at, runs = 0, []
    for (e, n), pad in zip(blocks_of, pads):
        end = at + 128 * n
        if n and e >= 0:
            index[at:end - pad] = e
            runs.append((at, end - pad, e))
        at = end
    return index, runs


# (experts, runs of (expert, 128-row blocks), padding rows at the end of each run)
CONTIGUOUS = [
    (1, [(0, 1)], [0]),
    (3, [(0, 1), (1, 2), (2, 1)], [5, 100, 127]),
    (4, [(0, 3), (2, 1), (3, 4)], [0, 64, 1]),                    # expert 1 empty
    (5, [(-1, 2), (4, 3), (-1, 1), (0, 2)], [0, 30, 0, 0]),       # blocks of padding
]


@pytest.mark.parametrize("case", range(len(CONTIGUOUS)))
@pytest.mark.parametrize("n,k", [(100, 384), (512, 256), (4100, 128)])
def test_contiguous_product(case, n, k):
    g, blocks_of, pads = CONTIGUOUS[case]
    _say(f"[gpu] contiguous mxfp4 case {case} n={n} k={k}")
    rng = np.random.default_rng(case * 10 + n)
    index, runs = contiguous_layout(rng, blocks_of, pads)
    m = index.size
    ca, ea, a = matrix(rng, (m, k))
    ea[index < 0] = 255                                            # padding rows are NaN
    cb, eb, b = matrix(rng, (g, n, k))
    d = torch.full((m, n), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_grouped_contiguous_nt_mxfp4(*pack(ca, ea), *pack(cb, eb), d,
                                            torch.from_numpy(index).cuda())
    for lo, hi, e in runs:
        err, want = product_bound(a[lo:hi], b[e])
        near(d[lo:hi], want, rounded(want, err), f"rows {lo}..{hi} of expert {e}")
    assert (d[torch.from_numpy(index < 0)] == SENTINEL).all()


MASKED = [(1, 1, [1]), (4, 96, [0, 96, 17, 500]), (3, 130, [129, 0, 128]), (2, 300, [257, 33]),
          (5, 16, [0, 0, 0, 0, 0]), (6, 70, [-3, 1, 2, 64, 65, 70])]


@pytest.mark.parametrize("case", range(len(MASKED)))
@pytest.mark.parametrize("n,k,expected", [(100, 384, 0), (1040, 256, 16), (384, 1152, 300)])
def test_masked_product(case, n, k, expected):
    g, max_m, masked = MASKED[case]
    _say(f"[gpu] masked mxfp4 case {case} n={n} k={k} expected={expected}")
    rng = np.random.default_rng(case * 10 + n)
    ca, ea, a = matrix(rng, (g, max_m, k))
    count = np.clip(masked, 0, max_m)
    for i in range(g):
        ea[i, count[i]:] = 255
    cb, eb, b = matrix(rng, (g, n, k))
    d = torch.full((g, max_m, n), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_grouped_masked_nt_mxfp4(*pack(ca, ea), *pack(cb, eb), d,
                                        torch.tensor(masked, dtype=torch.int32, device="cuda"),
                                        expected_m=expected)
    for i in range(g):
        c = count[i]
        err, want = product_bound(a[i, :c], b[i])
        near(d[i, :c], want, rounded(want, err), f"slot {i}")
        assert (d[i, c:] == SENTINEL).all()


# ---- gated block ---------------------------------------------------------------

GATED = [(1, 32, 128), (5, 96, 384), (64, 128, 256), (70, 416, 640), (130, 160, 128),
         (300, 1056, 256), (1030, 2080, 128)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,f,k", GATED)
def test_gated_dense(m, f, k, act):
    _say(f"[gpu] gated dense {m} {f} {k} {act}")
    rng = np.random.default_rng(m + f + k)
    ca, ea, a = matrix(rng, (m, k))
    cb, eb, b = matrix(rng, (2 * f, k), 2.0 / np.sqrt(k))
    h = torch.full((m + 1, f), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_gated_dense_mxfp4(*pack(ca, ea), *pack(cb, eb), h[:m], activation=act)
    want, err = gated_bound(a, b, f, act)
    near(h[:m], want, rounded(want, err), f"gated {m}x{f}x{k}")
    assert (h[m] == SENTINEL).all()


@pytest.mark.parametrize("case", range(len(CONTIGUOUS)))
def test_gated_contiguous(case):
    g, blocks_of, pads = CONTIGUOUS[case]
    f, k = 224, 384
    rng = np.random.default_rng(case)
    index, runs = contiguous_layout(rng, blocks_of, pads)
    ca, ea, a = matrix(rng, (index.size, k))
    ea[index < 0] = 255
    cb, eb, b = matrix(rng, (g, 2 * f, k), 2.0 / np.sqrt(k))
    h = torch.full((index.size, f), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_gated_contiguous_mxfp4(*pack(ca, ea), *pack(cb, eb), h,
                                       torch.from_numpy(index).cuda())
    for lo, hi, e in runs:
        want, err = gated_bound(a[lo:hi], b[e], f, "silu")
        near(h[lo:hi], want, rounded(want, err), f"expert {e}")
    assert (h[torch.from_numpy(index < 0)] == SENTINEL).all()


def check_quantised(hq, sfh, rows, want, err, what):
    """hq, sfh stand for a quantisation of some h within err of want: the exponent is that of
    one of the two ends of the largest magnitude's interval, each value no further from want
    than half a step plus err (or saturated)."""
    code, e, _ = unpack(hq, sfh, rows)
    got = values(code, e)
    b = np.abs(want).reshape(rows, -1, 32)
    eb = err.reshape(rows, -1, 32)
    lo, hi = (b - eb).max(-1), (b + eb).max(-1)
    lo_e = np.floor(np.log2(np.maximum(lo, 1e-300))) - 2
    hi_e = np.floor(np.log2(np.maximum(hi, 1e-300))) - 2
    sh = e.astype(np.float64) - 127
    assert ((sh >= np.maximum(lo_e, -127)) & (sh <= np.maximum(hi_e, -127))).all(), what
    s = 2.0 ** np.repeat(sh, 32, -1)
    top = np.abs(want) / s
    step = np.where(top < 2, 0.5, np.where(top < 4, 1.0, 2.0))
    room = np.where(top > 6, top - 6, 0) + step / 2
    bad = np.abs(got - want) > room * s + err * (1 + 1e-6) + 1e-300
    # an error that moves a value over a step's edge doubles the step there
    edge = np.abs(got - want) > room * s * 2 + err * (1 + 1e-6)
    assert bad.mean() < 1e-4 and not edge.any(), what


@pytest.mark.parametrize("m,f,k", [(1, 128, 128), (37, 256, 384), (130, 640, 256), (300, 2176, 128)])
def test_gated_quantised_output(m, f, k):
    _say(f"[gpu] gated dense quantised {m} {f} {k}")
    rng = np.random.default_rng(m + f)
    ca, ea, a = matrix(rng, (m, k))
    cb, eb, b = matrix(rng, (2 * f, k), 2.0 / np.sqrt(k))
    hq = torch.full((m, f // 2), 0xAB, dtype=torch.uint8, device="cuda")
    sfh = torch.full((f // 128, fp8bs.get_sfa_ld(m)), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    fp8bs.fp8bs_gated_dense_mxfp4_q(*pack(ca, ea), *pack(cb, eb), hq, sfh, activation="gelu_tanh")
    want, err = gated_bound(a, b, f, "gelu_tanh")
    check_quantised(hq, sfh, m, want, err, f"{m}x{f}x{k}")
    assert (unpack(hq, sfh, m)[2] == 0x5A).all()


def test_quantised_output_of_nan_and_zero_rows():
    m, f, k = 40, 128, 256
    rng = np.random.default_rng(1)
    ca, ea, a = matrix(rng, (m, k))
    ca[3] = 0                                             # h = act(0) * 0 = 0
    ea[7, 2] = 255                                        # the row is not a number
    cb, eb, b = matrix(rng, (2 * f, k), 0.1)
    hq = torch.empty(m, f // 2, dtype=torch.uint8, device="cuda")
    sfh = torch.empty(1, 40, dtype=torch.int32, device="cuda")
    fp8bs.fp8bs_gated_dense_mxfp4_q(*pack(ca, ea), *pack(cb, eb), hq, sfh)
    code, e, _ = unpack(hq, sfh, m)
    assert (e[3] == 0).all() and (code[3] % 8 == 0).all()
    assert (e[7] == 255).all() and (code[7] == 0).all()
    assert (np.delete(e, [3, 7], 0) < 200).all()


@pytest.mark.parametrize("case", range(len(MASKED)))
def test_gated_masked(case):
    g, max_m, masked = MASKED[case]
    f, k = 256, 384
    rng = np.random.default_rng(case)
    count = np.clip(masked, 0, max_m)
    ca, ea, a = matrix(rng, (g, max_m, k))
    for i in range(g):
        ea[i, count[i]:] = 255
    cb, eb, b = matrix(rng, (g, 2 * f, k), 2.0 / np.sqrt(k))
    ops = pack(ca, ea) + pack(cb, eb)
    mm = torch.tensor(masked, dtype=torch.int32, device="cuda")
    h = torch.full((g, max_m, f), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_gated_masked_mxfp4(*ops, h, mm, expected_m=40, activation="gelu_tanh")
    hq = torch.full((g, max_m, f // 2), 0xAB, dtype=torch.uint8, device="cuda")
    ld = fp8bs.get_sfa_ld(max_m)
    sfh = torch.full((g, f // 128, ld), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    fp8bs.fp8bs_gated_masked_mxfp4_q(*ops, hq, sfh, mm, expected_m=40, activation="gelu_tanh")
    for i in range(g):
        c = count[i]
        assert (h[i, c:] == SENTINEL).all() and (hq[i, c:] == 0xAB).all()
        assert (unpack(hq[i], sfh[i], c)[2] == 0x5A).all()
        if c:
            want, err = gated_bound(a[i, :c], b[i], f, "gelu_tanh")
            near(h[i, :c], want, rounded(want, err), f"slot {i}")
            check_quantised(hq[i, :c], sfh[i], c, want, err, f"slot {i}")


# ---- backward ------------------------------------------------------------------

def backward_bounds(x, w, f, dh, act):
    """(da, its bound, db, its bound): dg and du are rounded to bf16 (U), the recomputed
    projections carry the FP32 sums' error, then FP32 sums and one rounding."""
    eg, g = product_bound(x, w[:f])
    eu, u = product_bound(x, w[f:])
    v, s = _act(g, act)
    # |act''| <= 1.2 bounds the slope's change, |act'| <= 1.13 the value's
    es = 1.2 * eg + (32 + 2 * np.abs(g)) * E
    ev = 1.13 * eg + (16 + np.abs(g)) * E * np.maximum(np.abs(v), np.abs(g) * 2.0 ** -20)
    dg, du = dh * u * s, dh * v
    edg = np.abs(dh) * (np.abs(u) * es + np.abs(s) * eu + es * eu) + (U + 8 * E) * np.abs(dg)
    edu = np.abs(dh) * ev + (U + 8 * E) * np.abs(du)
    edg *= 1 + U
    edu *= 1 + U
    d, ed = np.concatenate((dg, du), 1), np.concatenate((edg, edu), 1)
    da = d @ w
    db = d.T @ x
    bda = ed @ np.abs(w) + (2 * f + 8) * E * (np.abs(d) @ np.abs(w))
    bdb = ed.T @ np.abs(x) + (x.shape[0] + 8) * E * (np.abs(d).T @ np.abs(x))
    return da, rounded(da, bda), db, rounded(db, bdb)


BACKWARD = [(1, 32, 128), (5, 64, 256), (64, 96, 384), (129, 160, 128), (200, 416, 640),
            (300, 256, 1152), (1100, 1056, 256)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,f,k", BACKWARD)
def test_backward_dense(m, f, k, act):
    _say(f"[gpu] gated backward {m} {f} {k} {act}")
    rng = np.random.default_rng(m + f + k)
    ca, ea, a = matrix(rng, (m, k))
    cb, eb, b = matrix(rng, (2 * f, k), 2.0 / np.sqrt(k))
    dh = bf16(rng.standard_normal((m, f)))
    da, bda, db, bdb = backward_bounds(a, b, f, dh.double().numpy(), act)
    ops = pack(ca, ea, 255) + pack(cb, eb, 255) + (dh.cuda(),)
    ga = torch.full((m + 1, k), SENTINEL, dtype=torch.bfloat16, device="cuda")
    gb = torch.full((2 * f, k), SENTINEL, dtype=torch.bfloat16, device="cuda")
    size = fp8bs.gated_backward_workspace_size(fp8bs.LAYOUT_DENSE, m, f, k)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")   # NaNs if any were read
    fp8bs.fp8bs_gated_dense_mxfp4_backward(*ops, ga[:m], gb, activation=act, workspace=ws)
    near(ga[:m], da, bda, "da")
    near(gb, db, bdb, "db")
    assert (ga[m] == SENTINEL).all()
    # each alone, and the FP32 form with what it adds to
    only = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_gated_dense_mxfp4_backward(*ops, only, None, activation=act)
    assert torch.equal(only, ga[:m])
    start = torch.randn(2 * f, k, device="cuda")
    full = start.clone()
    fp8bs.fp8bs_gated_dense_mxfp4_backward(*ops, None, full, activation=act, accumulate=True)
    plain = torch.empty_like(full)
    fp8bs.fp8bs_gated_dense_mxfp4_backward(*ops, None, plain, activation=act)
    assert torch.equal(plain.bfloat16(), gb)
    assert torch.equal(full, start + plain)


# few tiles of a long contraction, in parts: db's (tokens), da's (columns of W), both
@pytest.mark.parametrize("m,f,k", [(2085, 64, 256), (70, 1056, 128), (1300, 704, 128)])
def test_backward_in_parts(m, f, k):
    test_backward_dense(m, f, k, "silu")


@pytest.mark.parametrize("case", range(len(CONTIGUOUS)))
@pytest.mark.parametrize("f,k", [(96, 256), (640, 1152)])
def test_backward_contiguous(case, f, k):
    g, blocks_of, pads = CONTIGUOUS[case]
    _say(f"[gpu] gated backward contiguous case {case} f={f} k={k}")
    rng = np.random.default_rng(case + f)
    index, runs = contiguous_layout(rng, blocks_of, pads)
    m = index.size
    ca, ea, a = matrix(rng, (m, k))
    ea[index < 0] = 255
    cb, eb, b = matrix(rng, (g, 2 * f, k), 2.0 / np.sqrt(k))
    dh = bf16(rng.standard_normal((m, f)))
    dh[torch.from_numpy(index < 0)] = float("nan")
    ga = torch.full((m, k), SENTINEL, dtype=torch.bfloat16, device="cuda")
    gb = torch.full((g, 2 * f, k), SENTINEL, dtype=torch.float32, device="cuda")
    size = fp8bs.gated_backward_workspace_size(fp8bs.LAYOUT_CONTIGUOUS, m, f, k, g)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    layout = torch.from_numpy(index).cuda()
    ops = pack(ca, ea) + pack(cb, eb) + (dh.cuda(),)
    fp8bs.fp8bs_gated_contiguous_mxfp4_backward(*ops, ga, gb, layout, workspace=ws)
    seen = set()
    for lo, hi, e in runs:
        seen.add(e)
        da, bda, db, bdb = backward_bounds(a[lo:hi], b[e], f, dh[lo:hi].double().numpy(), "silu")
        near(ga[lo:hi], da, bda, f"da of expert {e}")
        near(gb[e], db, bdb, f"db of expert {e}")
    for e in set(range(g)) - seen:
        assert (gb[e] == 0).all()
    assert (ga[torch.from_numpy(index < 0)] == SENTINEL).all()
    again = torch.empty_like(gb)
    fp8bs.fp8bs_gated_contiguous_mxfp4_backward(*ops, None, again, layout)
    assert torch.equal(again, gb)


def test_gradient_against_differences():
    # The loss sum(dh * h), as a 64-bit function of the values that codes and exponents stand
    # for, along random directions: its central difference against the gradients' projection.
    # Step 1e-5: the difference errs by 1e-10 of third derivatives and 1e-11 of the loss's
    # rounding, far below the kernels' own bound.
    m, f, k = 24, 64, 128
    rng = np.random.default_rng(77)
    ca, ea, a = matrix(rng, (m, k))
    cb, eb, b = matrix(rng, (2 * f, k), 2.0 / np.sqrt(k))
    dh = bf16(rng.standard_normal((m, f)))
    d64 = dh.double().numpy()
    ga = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    gb = torch.empty(2 * f, k, dtype=torch.float32, device="cuda")
    fp8bs.fp8bs_gated_dense_mxfp4_backward(*pack(ca, ea), *pack(cb, eb), dh.cuda(), ga, gb)

    def loss(x, w):
        return (d64 * _act(x @ w[:f].T, "silu")[0] * (x @ w[f:].T)).sum()

    _, bda, _, bdb = backward_bounds(a, b, f, d64, "silu")
    for _ in range(4):
        da, db = rng.standard_normal(a.shape), rng.standard_normal(b.shape)
        h = 1e-5
        num = (loss(a + h * da, b) - loss(a - h * da, b)) / (2 * h)
        got = (ga.cpu().double().numpy() * da).sum()
        assert abs(num - got) <= (bda * np.abs(da)).sum() + 1e-6 * abs(num)
        num = (loss(a, b + h * db) - loss(a, b - h * db)) / (2 * h)
        got = (gb.cpu().double().numpy() * db).sum()
        assert abs(num - got) <= (bdb * np.abs(db)).sum() + 1e-6 * abs(num)


@pytest.mark.parametrize("layout", ["dense", "contiguous"])
def test_gradients_together_are_the_gradients_alone(layout):
    # both in one launch (contiguous: of more 128x128 tiles, 16 x 8 + 16 x 8 for each of five
    # experts, than run at once) against one after the other: every sum has the same order
    rng = np.random.default_rng(61)
    m, f, k, g = 2048, 1024, 1024, 5
    lead = () if layout == "dense" else (g,)
    a, b = pack(*matrix(rng, (m, k))[:2]), pack(*matrix(rng, lead + (2 * f, k), 0.1)[:2])
    dh = bf16(rng.standard_normal((m, f))).cuda()
    extra = () if layout == "dense" else (
        torch.arange(m // 128, dtype=torch.int32).mul(7).remainder(g).repeat_interleave(128).cuda(),)
    call = getattr(fp8bs, f"fp8bs_gated_{layout}_mxfp4_backward")
    da, da2 = (torch.zeros(m, k, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    db, db2 = (torch.zeros(*lead, 2 * f, k, device="cuda") for _ in range(2))
    call(*a, *b, dh, da, db, *extra)
    call(*a, *b, dh, da2, None, *extra)
    call(*a, *b, dh, None, db2, *extra)
    assert torch.equal(da, da2) and torch.equal(db, db2)
    assert bool(da.any(1).all()) and bool(db.any(-1).all())


def test_backward_in_parts_contiguous():
    # experts of 42, 0 and 10 steps in two parts each; the middle one's are both empty
    rng = np.random.default_rng(62)
    f, k, g = 64, 256, 3
    index, runs = contiguous_layout(rng, [(0, 21), (2, 5)], [3, 100])
    ca, ea, a = matrix(rng, (index.size, k))
    cb, eb, b = matrix(rng, (g, 2 * f, k), 2.0 / np.sqrt(k))
    dh = bf16(rng.standard_normal((index.size, f)))
    dh[torch.from_numpy(index < 0)] = float("nan")
    start = torch.randn(g, 2 * f, k, device="cuda")
    gb, plain = start.clone(), torch.empty_like(start)
    size = fp8bs.gated_backward_workspace_size(fp8bs.LAYOUT_CONTIGUOUS, index.size, f, k, g)
    ops = pack(ca, ea) + pack(cb, eb) + (dh.cuda(), None)
    layout = torch.from_numpy(index).cuda()
    for out, add in ((plain, False), (gb, True)):
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        fp8bs.fp8bs_gated_contiguous_mxfp4_backward(*ops, out, layout, accumulate=add, workspace=ws)
    for lo, hi, e in runs:
        _, _, db, bdb = backward_bounds(a[lo:hi], b[e], f, dh[lo:hi].double().numpy(), "silu")
        near(plain[e], db, bdb, f"db of expert {e}")
    assert (plain[1] == 0).all()
    assert torch.equal(gb, start + plain)


def test_k_past_32_bits_is_refused():
    # (a call's k is an int: 2^32 + 256 would pass as 256)
    k = (1 << 32) + 256
    q = torch.empty(1, k // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(k // 128, 4, dtype=torch.int32, device="cuda")
    d = torch.full((1, 1), 5.0, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: fp8bs.fp8bs_dense_nt_mxfp4(q, sf, q, sf, d),
                 lambda: fp8bs.dequantize_mxfp4(q, sf),
                 lambda: fp8bs.quantize_mxfp4(q.view(torch.bfloat16)[:, :1 << 25])):
        with pytest.raises(fp8bs.FP8BSError):
            call()
    assert d.item() == 5.0


# ---- layer, streams, graphs ------------------------------------------------------

@pytest.mark.parametrize("layout", ["dense", "contiguous", "masked"])
def test_feed_forward_layer_is_its_parts(layout):
    rng = np.random.default_rng(4)
    f, k, g = 256, 384, 3
    lead = () if layout == "dense" else (g,)
    b, sfb = pack(*matrix(rng, lead + (2 * f, k), 0.1)[:2])
    b2, sfb2 = pack(*matrix(rng, lead + (k, f), 0.1)[:2])
    if layout == "masked":
        x = bf16(rng.standard_normal((g, 50, k))).cuda()
        extra = dict(masked_m=torch.tensor([50, 0, 7], dtype=torch.int32, device="cuda"))
        data = (extra["masked_m"],)
    elif layout == "contiguous":
        index, _ = contiguous_layout(rng, [(0, 1), (2, 2)], [3, 100])
        x = bf16(rng.standard_normal((index.size, k))).cuda()
        extra = dict(grouped_layout=torch.from_numpy(index).cuda())
        data = (extra["grouped_layout"],)
    else:
        x = bf16(rng.standard_normal((77, k))).cuda()
        extra, data = {}, ()
    out = torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda")
    assert fp8bs.feed_forward_mxfp4(x, b, sfb, b2, sfb2, out=out, **extra) is out
    q, sf = fp8bs.quantize_mxfp4(x)
    hq = torch.zeros(x.shape[:-1] + (f // 2,), dtype=torch.uint8, device="cuda")
    sfh = torch.zeros(x.shape[:-2] + (f // 128, fp8bs.get_sfa_ld(x.shape[-2])), dtype=torch.int32,
                      device="cuda")
    want = torch.zeros_like(out)
    name = {"dense": "dense", "contiguous": "contiguous", "masked": "masked"}[layout]
    getattr(fp8bs, f"fp8bs_gated_{name}_mxfp4_q")(q, sf, b, sfb, hq, sfh, *data)
    product = {"dense": fp8bs.fp8bs_dense_nt_mxfp4,
               "contiguous": fp8bs.fp8bs_grouped_contiguous_nt_mxfp4,
               "masked": fp8bs.fp8bs_grouped_masked_nt_mxfp4}[layout]
    product(hq, sfh, b2, sfb2, want, *data)
    assert torch.equal(out, want) and out.abs().sum() > 0


def test_calls_on_another_stream_and_repeated_in_a_graph():
    rng = np.random.default_rng(8)
    m, f, k = 60, 256, 384
    x = bf16(rng.standard_normal((m, k))).cuda()
    b, sfb = pack(*matrix(rng, (2 * f, k), 0.1)[:2])
    b2, sfb2 = pack(*matrix(rng, (k, f), 0.1)[:2])
    want = fp8bs.feed_forward_mxfp4(x, b, sfb, b2, sfb2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fp8bs.feed_forward_mxfp4(x, b, sfb, b2, sfb2, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    with torch.cuda.stream(side):
        fp8bs.feed_forward_mxfp4(x, b, sfb, b2, sfb2, out=out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8bs.feed_forward_mxfp4(x, b, sfb, b2, sfb2, out=out)
    for i in range(3):
        x.copy_(bf16(rng.standard_normal((m, k))))
        want = fp8bs.feed_forward_mxfp4(x, b, sfb, b2, sfb2)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"


@pytest.mark.parametrize("m", [0, 1, 2, 200])
def test_results_do_not_change_from_call_to_call(m):
    rng = np.random.default_rng(m)
    f, k = 96, 256
    ca, ea, _ = matrix(rng, (max(m, 1), k))
    cb, eb, _ = matrix(rng, (2 * f, k), 0.1)
    a, sfa = (pack(ca, ea) if m else (torch.empty(0, k // 2, dtype=torch.uint8, device="cuda"),
                                      torch.empty(2, 0, dtype=torch.int32, device="cuda")))
    b, sfb = pack(cb, eb)
    dh = torch.randn(m, f, device="cuda").bfloat16()
    runs = []
    for _ in range(2):
        d = torch.empty(m, 2 * f, dtype=torch.bfloat16, device="cuda")
        h = torch.empty(m, f, dtype=torch.bfloat16, device="cuda")
        da = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
        db = torch.full((2 * f, k), SENTINEL, device="cuda")
        fp8bs.fp8bs_dense_nt_mxfp4(a, sfa, b, sfb, d)
        fp8bs.fp8bs_gated_dense_mxfp4(a, sfa, b, sfb, h)
        fp8bs.fp8bs_gated_dense_mxfp4_backward(a, sfa, b, sfb, dh, da, db)
        runs.append((d, h, da, db))
    assert all(torch.equal(x, y) for x, y in zip(*runs))
    if m == 0:
        assert (runs[0][3] == 0).all()


# ---- every kernel, long lists, long operands ---------------------------------------

# rows and columns at which the few-rows kernel takes each of its tile shapes and the LDS
# kernel its two, with odd rests in every direction
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 33, 47, 64, 65, 100, 129, 250, 385, 700])
@pytest.mark.parametrize("n,k", [(31, 128), (130, 640), (1000, 896), (2112, 256), (4097, 384)])
def test_product_of_every_tile_shape(m, n, k):
    rng = np.random.default_rng(m * 7 + n)
    ca, ea, a = matrix(rng, (m, k))
    cb, eb, b = matrix(rng, (n, k))
    d = torch.full((m + 1, n), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_dense_nt_mxfp4(*pack(ca, ea, 255), *pack(cb, eb, 255), d[:m])
    err, want = product_bound(a, b)
    near(d[:m], want, rounded(want, err), f"{m}x{n}x{k}")
    assert (d[m] == SENTINEL).all()


@pytest.mark.parametrize("max_m,masked,expected", [
    (40, [40, 3, 0], 4), (90, [90, 1], 16), (300, [300, 0, 150, 17], 20), (64, [64], 64)])
@pytest.mark.parametrize("n,k", [(100, 384), (320, 1152)])
def test_slots_with_more_rows_than_expected(max_m, masked, expected, n, k):
    # the hint only steers the choice of kernel; slots with more rows are walked through
    rng = np.random.default_rng(max_m + n)
    g = len(masked)
    ca, ea, a = matrix(rng, (g, max_m, k))
    cb, eb, b = matrix(rng, (g, n, k))
    d = torch.full((g, max_m, n), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_grouped_masked_nt_mxfp4(*pack(ca, ea), *pack(cb, eb), d,
                                        torch.tensor(masked, dtype=torch.int32, device="cuda"),
                                        expected_m=expected)
    for i, c in enumerate(masked):
        err, want = product_bound(a[i, :c], b[i])
        near(d[i, :c], want, rounded(want, err), f"slot {i}")
        assert (d[i, c:] == SENTINEL).all()


def _few(rng, total, few):
    """a packed operand of `total` rows of 128 values, of which only `few` are not zero"""
    code = np.zeros((len(few), 128), np.uint8)
    code[:] = rng.integers(0, 16, code.shape)
    e = rng.integers(120, 130, (len(few), 4)).astype(np.uint8)
    q, sf = pack(code, e)
    full_q = torch.zeros(total, 64, dtype=torch.uint8, device="cuda")
    full_sf = torch.zeros(1, fp8bs.get_sfa_ld(total), dtype=torch.int32, device="cuda")
    at = torch.tensor(few, device="cuda")
    full_q[at] = q
    full_sf[0, at] = sf[0, :len(few)]
    return full_q, full_sf, values(code, e)


def test_more_tiles_than_one_launch_lists():
    # contiguous: 2050 blocks of 128 rows (a launch lists 2048), runs crossing the limit
    rng = np.random.default_rng(21)
    blocks, g, n, f = 2050, 3, 48, 32
    few = [0, 127, 128, 2047 * 128 + 5, 2048 * 128, 2048 * 128 + 127, 2049 * 128 + 64]
    a, sfa, va = _few(rng, blocks * 128, few)
    index = np.full(blocks * 128, -1, np.int32)
    index[:1000 * 128 + 77] = 0
    index[1001 * 128:2049 * 128] = 2
    index[2049 * 128:2049 * 128 + 100] = 1
    layout = torch.from_numpy(index).cuda()
    cb, eb, b = matrix(rng, (g, n, 128))
    d = torch.full((blocks * 128, n), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_grouped_contiguous_nt_mxfp4(a, sfa, *pack(cb, eb), d, layout)
    want = np.zeros((len(few), n))
    err = np.zeros_like(want)
    for i, r in enumerate(few):
        err[i], want[i] = (x[0] for x in product_bound(va[i:i + 1], b[index[r]]))
    near(d[torch.tensor(few, device="cuda")], want, rounded(want, err), "rows")
    valid = layout >= 0
    assert (d[~valid] == SENTINEL).all()
    zero = valid.clone()
    zero[torch.tensor(few, device="cuda")] = False
    assert (d[zero] == 0).all()
    # and the backward pass over them
    cb, eb, b = matrix(rng, (g, 2 * f, 128), 0.1)
    dh = torch.zeros(blocks * 128, f, dtype=torch.bfloat16, device="cuda")
    rows = bf16(rng.standard_normal((len(few), f)))
    dh[torch.tensor(few, device="cuda")] = rows.cuda()
    da = torch.full((blocks * 128, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
    db = torch.full((g, 2 * f, 128), SENTINEL, device="cuda")
    fp8bs.fp8bs_gated_contiguous_mxfp4_backward(a, sfa, *pack(cb, eb), dh, da, db, layout)
    for e in range(g):
        mine = [i for i, r in enumerate(few) if index[r] == e]
        wa, ba, wb, bb = backward_bounds(va[mine], b[e], f, rows.double().numpy()[mine], "silu")
        near(da[torch.tensor([few[i] for i in mine], device="cuda")], wa, ba, f"da of expert {e}")
        near(db[e], wb, bb, f"db of expert {e}")
    assert (da[zero] == 0).all() and (da[~valid] == SENTINEL).all()


def test_more_slots_than_one_launch_lists():
    g, max_m, n, k = 2100, 130, 16, 128
    rng = np.random.default_rng(5)
    code = torch.from_numpy(rng.integers(0, 256, (g, max_m, k // 2)).astype(np.uint8)).cuda()
    sf = torch.full((g, 1, fp8bs.get_sfa_ld(max_m)), 0x7F7F7F7F, dtype=torch.int32, device="cuda")
    cb, eb, b = matrix(rng, (g, n, k))
    masked = rng.integers(0, max_m + 1, g).astype(np.int32)
    d = torch.full((g, max_m, n), float("inf"), dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_grouped_masked_nt_mxfp4(code, sf, *pack(cb, eb), d, torch.from_numpy(masked).cuda(),
                                        expected_m=65)
    q = code.cpu().numpy()
    v = E2M1[np.stack((q & 15, q >> 4), -1).reshape(g, max_m, k)]
    for i in (0, 1, 1023, 1024, 2047, 2048, 2099):
        c = masked[i]
        err, want = product_bound(v[i, :c], b[i])
        near(d[i, :c], want, rounded(want, err), f"slot {i}")
    rows = torch.arange(max_m, device="cuda")[None] >= torch.from_numpy(masked).cuda()[:, None]
    assert torch.isinf(d[rows]).all() and torch.isfinite(d[~rows]).all()


def test_operands_past_four_gigabytes():
    # 4.6 GB of codes: the last rows' addresses need more than 32 bits
    m, n, k = 560_003, 24, 16384
    rng = np.random.default_rng(2)
    a = torch.zeros(m, k // 2, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(k // 128, fp8bs.get_sfa_ld(m), dtype=torch.int32, device="cuda")
    tail = 70
    ca, ea, va = matrix(rng, (tail, k))
    q, sf = pack(ca, ea)
    a[m - tail:] = q
    sfa[:, m - tail:m] = sf[:, :tail]
    cb, eb, b = matrix(rng, (n, k))
    d = torch.full((m, n), SENTINEL, dtype=torch.bfloat16, device="cuda")
    fp8bs.fp8bs_dense_nt_mxfp4(a, sfa, *pack(cb, eb), d)
    err, want = product_bound(va, b)
    near(d[m - tail:], want, rounded(want, err), "last rows")
    assert (d[:m - tail] == 0).all()
    x = fp8bs.dequantize_mxfp4(a, sfa)                     # 18 GB
    assert np.array_equal(x[m - tail:].cpu().double().numpy(), va)
    q2, sf2 = fp8bs.quantize_mxfp4(x)
    y = fp8bs.dequantize_mxfp4(q2[m - tail:].contiguous(), sf2[:, m - tail:].contiguous()
                               if tail % 4 == 0 else _last(sf2, m, tail))
    assert np.array_equal(y.cpu().double().numpy(), va)


def _last(sf, m, tail):
    out = torch.zeros(sf.shape[0], fp8bs.get_sfa_ld(tail), dtype=torch.int32, device="cuda")
    out[:, :tail] = sf[:, m - tail:m]
    return out
