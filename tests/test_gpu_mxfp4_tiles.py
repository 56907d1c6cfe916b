"""GPU tests of the MXFP4 operators' kernels one by one against their definitions in 64 bits,
with the bounds that tests/test_gpu_mxfp4.py derives.

Which kernel a call launches is a cost model of its sizes.  The sizes of _mx_cases.py launch every
compiled one (tests/test_mxfp4_launches.py asserts it): the 256x256 and 128x128 tiles of every
layout and epilogue, masked lists, every few-rows tile, both gradient products by every tile, side
by side and in parts."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs
from _mx_cases import CASES, CONTIGUOUS, DENSE, MASKED
from test_gpu_mxfp4 import (_act, _say, backward_bounds, bf16, check_quantised, gated_bound, near, pack,
                            product_bound, quantise, rounded, unpack, values)

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
    with np.errstate(over="ignore"):
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


# ---- every kernel ----------------------------------------------------------------

SENTINEL = 77.0


def random_operand(rng, shape, low, high):
    """codes, exponents from 2^(low - 127) to 2^(high - 127)"""
    return (rng.integers(0, 16, shape, dtype=np.uint8),
            rng.integers(low, high + 1, shape[:-1] + (shape[-1] // 32,), dtype=np.uint8))


def slots(g, max_m):
    """rows that each slot holds (negative and too large ones among them)"""
    of = [max_m, 0, 1, 127, 128, 129, max_m - 1, 17, 255, 256, 257, -3, max_m + 200, 64, 65, 33]
    return [of[(i + i // 16) % 16] for i in range(g)]


def blocks(rng, m, g):
    """grouped_layout and [(start, end, expert)]: experts in any order, some without rows, blocks
    of padding, ragged ends"""
    n = m // 128
    order = rng.permutation(g)
    cuts = np.sort(rng.integers(0, n + 1, g - 1))
    if n == 1:
        order, cuts = np.arange(g), np.full(g - 1, n)
    index, runs = np.full(m, -1, np.int32), []
    for e, lo, hi in zip(order, [0, *cuts], [*cuts, n]):
        if hi - lo > 3:
            lo += 1                                       # a block of padding before the run
        if hi > lo:
            end = 128 * hi - int(rng.choice([0, 1, 63, 64, 100, 127]))
            index[128 * lo:end] = e
            runs.append((128 * lo, end, int(e)))
    return index, runs


def device(x):
    return torch.from_numpy(x).cuda()


def parts_of(layout, m, g, rng):
    """(extra argument, mask of rows that are not valid, [(where, expert)])"""
    if layout == DENSE:
        return None, None, [(slice(0, m), None)]
    if layout == CONTIGUOUS:
        index, runs = blocks(rng, m, g)
        return device(index), index < 0, [(slice(lo, hi), e) for lo, hi, e in runs]
    count = slots(g, m)
    held = np.clip(count, 0, m)
    which = range(g) if g < 100 else [*range(12), 1020, 1023, 1024, 2040, 2046, 2047, 2048, 2049, g - 2, g - 1]
    return (torch.tensor(count, dtype=torch.int32, device="cuda"),
            np.arange(m)[None] >= held[:, None], [((i, slice(0, held[i])), i) for i in which if held[i]])


@pytest.mark.parametrize("case", range(len(CASES)), ids=lambda i: "-".join(map(str, CASES[i])))
def test_every_kernel_against_the_definition(case):
    op, layout, m, expected, n, k, g, flag = CASES[case]
    _say(f"[gpu] {CASES[case]}")
    rng = np.random.default_rng(1000 + case)
    if op in ("quantise", "dequantise"):
        x = torch.from_numpy(rng.standard_normal((g, m, k)).astype(np.float32)).to(
            torch.bfloat16 if flag else torch.float32)
        code, e = quantise(x.double().numpy())
        q, sf = fp8bs.quantize_mxfp4(x.cuda())
        if op == "quantise":
            got, exponents, _ = unpack(q, sf, m)
            assert np.array_equal(got, code) and np.array_equal(exponents, e)
        else:
            y = fp8bs.dequantize_mxfp4(q, sf, x.dtype)
            assert y.dtype == x.dtype and np.array_equal(y.cpu().double().numpy(), values(code, e))
        return
    extra, void, parts = parts_of(layout, m, g, rng)
    data = () if extra is None else (extra,)
    hint = dict(expected_m=expected) if layout == MASKED else {}
    name = ("dense", "contiguous", "masked")[layout]
    rows = (g, m) if layout == MASKED else (m,)
    lead = () if layout == DENSE else (g,)
    act = "gelu_tanh" if case % 2 else "silu"
    cols = n if op == "product" else 2 * n
    # products of gates and ups of about 1, from sums of k terms of every size
    ca, ea = random_operand(rng, rows + (k,), 121, 126)
    top = 124 - int(np.log2(k) / 2)
    cb, eb = random_operand(rng, lead + (cols, k), top - 3, top)
    if void is not None:
        ea[void] = 255                                     # what no row holds is not a number
    ops = pack(ca, ea, 255) + pack(cb, eb, 255)

    def at(where, e):
        return values(ca[where], ea[where]), values(cb[e], eb[e]) if lead else values(cb, eb)

    def untouched(out, mark):
        if layout == DENSE:
            return bool((out[-1] == mark).all())           # a row past the last one
        return bool((out[device(void)] == mark).all())

    spare = rows if layout != DENSE else (m + 1,)

    def cut(out):
        return out[:m] if layout == DENSE else out

    if op == "product":
        d = torch.full(spare + (n,), SENTINEL, dtype=torch.bfloat16, device="cuda")
        call = "fp8bs_dense_nt_mxfp4" if layout == DENSE else f"fp8bs_grouped_{name}_nt_mxfp4"
        getattr(fp8bs, call)(*ops, cut(d), *data, **hint)
        for where, e in parts:
            err, want = product_bound(*at(where, e))
            near(d[where], want, rounded(want, err), f"{where}")
        assert untouched(d, SENTINEL)
    elif op == "gated":
        h = torch.full(spare + (n,), SENTINEL, dtype=torch.bfloat16, device="cuda")
        getattr(fp8bs, f"fp8bs_gated_{name}_mxfp4")(*ops, cut(h), *data, activation=act, **hint)
        for where, e in parts:
            want, err = gated_bound(*at(where, e), n, act)
            near(h[where], want, rounded(want, err), f"{where}")
        assert untouched(h, SENTINEL)
    elif op == "gated_q":
        hq = torch.full(spare + (n // 2,), 0xAB, dtype=torch.uint8, device="cuda")
        sfh = torch.full(rows[:-1] + (n // 128, fp8bs.get_sfa_ld(m)), 0x5A5A5A5A, dtype=torch.int32,
                         device="cuda")
        getattr(fp8bs, f"fp8bs_gated_{name}_mxfp4_q")(*ops, cut(hq), sfh, *data, activation=act, **hint)
        for where, e in parts:
            want, err = gated_bound(*at(where, e), n, act)
            words = sfh[where[0]] if layout == MASKED else sfh
            span = where[1] if layout == MASKED else where
            count = span.stop - span.start
            own = torch.zeros(n // 128, fp8bs.get_sfa_ld(count), dtype=torch.int32, device="cuda")
            own[:, :count] = words[:, span]
            check_quantised(hq[where], own, count, want, err, f"{where}")
        assert untouched(hq, 0xAB)
        words = sfh.transpose(-1, -2)                      # [.., ld, n / 128]
        assert bool((words[..., m:, :] == 0x5A5A5A5A).all())
        if void is not None:
            assert bool((words[..., :m, :][device(void)] == 0x5A5A5A5A).all())
    else:
        f32, add = bool(flag & 4), bool(flag & 8)
        dh = bf16(rng.standard_normal((m, n)))
        if void is not None:
            dh[torch.from_numpy(void)] = float("nan")
        da = torch.full((m + 1, k), SENTINEL, dtype=torch.bfloat16, device="cuda") if flag & 1 else None
        db = torch.full(lead + (2 * n, k), SENTINEL, dtype=torch.float32 if f32 else torch.bfloat16,
                        device="cuda") if flag & 2 else None
        size = fp8bs.gated_backward_workspace_size(layout, m, n, k, g, bool(flag & 1), bool(flag & 2))
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")   # NaNs if any were read
        getattr(fp8bs, f"fp8bs_gated_{name}_mxfp4_backward")(
            *ops, dh.cuda(), None if da is None else da[:m], db, *data, activation=act, accumulate=add,
            workspace=ws)
        seen = set()
        for where, e in parts:
            wa, ba, wb, bb = backward_bounds(*at(where, e), n, dh[where].double().numpy(), act)
            if da is not None:
                near(da[where], wa, ba, f"da {where}")
            if db is not None:
                near(db[e] if lead else db, wb, bb, f"db {where}")
            seen.add(e)
        if db is not None and lead:
            assert all(bool((db[e] == 0).all()) for e in set(range(g)) - seen)
        if da is not None:
            assert bool((da[m] == SENTINEL).all())
            assert layout == DENSE or bool((da[:m][device(void)] == SENTINEL).all())


# ---- the layer -------------------------------------------------------------------

def quantised_range(h, err):
    """middle and half width of what the quantisation of a value within err of h may stand for"""
    b, eb = h.reshape(*h.shape[:-1], -1, 32), err.reshape(*h.shape[:-1], -1, 32)
    low = high = None
    for top in (np.abs(b) - eb, np.abs(b) + eb):
        amax = np.maximum(top.max(-1, keepdims=True), 0)
        e = np.floor(np.log2(np.where(amax > 0, amax, 2.0 ** -200))) - 2
        scale = 2.0 ** np.maximum(e, -127)
        for x in (b - eb, b + eb):
            a = np.abs(x) / scale
            step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
            v = np.sign(x) * np.minimum(np.round(a / step) * step, 6.0) * scale    # ties to even
            low = v if low is None else np.minimum(low, v)
            high = v if high is None else np.maximum(high, v)
    return ((low + high) / 2).reshape(h.shape), ((high - low) / 2).reshape(h.shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout,m,expected,f,k,n,g", [
    (DENSE, 77, 0, 256, 384, 201, 1), (DENSE, 1, 0, 128, 128, 30, 1), (DENSE, 700, 0, 640, 256, 300, 1),
    (CONTIGUOUS, 1152, 0, 256, 384, 200, 4), (MASKED, 50, 9, 256, 384, 200, 5),
    (MASKED, 300, 0, 384, 640, 210, 18)])
def test_layer_against_the_definition(layout, m, expected, f, k, n, g, dtype):
    _say(f"[gpu] layer {layout} {m} {f} {k} {n} {g} {dtype}")
    rng = np.random.default_rng(m + f)
    extra, void, parts = parts_of(layout, m, g, rng)
    rows = (g, m) if layout == MASKED else (m,)
    lead = () if layout == DENSE else (g,)
    x = torch.from_numpy(rng.standard_normal(rows + (k,)).astype(np.float32)).to(dtype)
    if void is not None:
        x[torch.from_numpy(void)] = float("nan")
    top = 124 - int(np.log2(k) / 2)
    cb, eb = random_operand(rng, lead + (2 * f, k), top - 3, top)
    c2, e2 = random_operand(rng, lead + (n, f), 118, 121)
    out = torch.full(rows + (n,), SENTINEL, dtype=torch.bfloat16, device="cuda")
    data = {DENSE: {}, CONTIGUOUS: dict(grouped_layout=extra),
            MASKED: dict(masked_m=extra, expected_m=expected)}[layout]
    fp8bs.feed_forward_mxfp4(x.cuda(), *pack(cb, eb, 255), *pack(c2, e2, 255), activation="gelu_tanh",
                             out=out, **data)
    xd = x.double().numpy()
    for where, e in parts:
        w, w2 = (values(cb[e], eb[e]), values(c2[e], e2[e])) if lead else (values(cb, eb), values(c2, e2))
        h, err = gated_bound(values(*quantise(xd[where])), w, f, "gelu_tanh")
        mid, half_width = quantised_range(h, err)
        err, want = product_bound(np.abs(mid) + half_width, w2)
        want = mid @ w2.T
        near(out[where], want, rounded(want, err + half_width @ np.abs(w2).T), f"{where}")
    if void is not None:
        assert bool((out[device(void)] == SENTINEL).all())


def test_codes_of_the_packed_type():
    # torch's type of two 4-bit values to a byte in place of uint8, everywhere codes are taken
    packed = getattr(torch, "float4_e2m1fn_x2", None)
    if packed is None:
        pytest.skip("this torch has no such type")
    rng = np.random.default_rng(3)
    m, f, k, n = 40, 128, 256, 70
    x = bf16(rng.standard_normal((m, k))).cuda()
    q, sf = fp8bs.quantize_mxfp4(x)
    q4 = torch.zeros_like(q).view(packed)
    sf4 = torch.empty_like(sf)
    fp8bs.fp8bs_quantize_mxfp4(x, q4, sf4)
    assert torch.equal(q4.view(torch.uint8), q)
    assert torch.equal(fp8bs.dequantize_mxfp4(q4, sf), fp8bs.dequantize_mxfp4(q, sf))
    b, sfb = pack(*random_operand(rng, (2 * f, k), 118, 121), 255)
    b2, sfb2 = pack(*random_operand(rng, (n, f), 118, 121), 255)
    dh = bf16(rng.standard_normal((m, f))).cuda()
    outs = []
    for view in (lambda t: t, lambda t: t.view(packed)):
        d = torch.empty(m, 2 * f, dtype=torch.bfloat16, device="cuda")
        fp8bs.fp8bs_dense_nt_mxfp4(view(q), sf, view(b), sfb, d)
        hq = torch.empty(m, f // 2, dtype=torch.uint8, device="cuda")
        sfh = torch.zeros(f // 128, m, dtype=torch.int32, device="cuda")
        fp8bs.fp8bs_gated_dense_mxfp4_q(view(q), sf, view(b), sfb, view(hq), sfh)
        da = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
        fp8bs.fp8bs_gated_dense_mxfp4_backward(view(q), sf, view(b), sfb, dh, da, None)
        y = fp8bs.feed_forward_mxfp4(x, view(b), sfb, view(b2), sfb2)
        outs.append((d, hq, sfh, da, y))
    assert all(torch.equal(one, other) for one, other in zip(*outs))
