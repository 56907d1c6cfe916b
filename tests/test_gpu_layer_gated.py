"""GPU tests of the gated activation with e4m3 output and checkpoint, of its backward pass and of the
quantiser along tokens, against their definitions in 64 bits.  What is one rounding after another of
given values (the checkpoint, columns, a value times its scale) is compared bit for bit; what passes
through the activation within the bounds that tests/_layer_ref.py derives for it and one FP32
rounding for each product."""
import itertools

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs
import _layer_ref as ref
from _layer_ref import E, host

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
NAN = float("nan")


@pytest.fixture
def gen():
    return torch.Generator("cuda").manual_seed(31)


def rand(gen, *shape, dtype=BF16, size=1.0):
    x = torch.randn(shape, generator=gen, device="cuda") * size
    return (x * torch.exp(torch.randn(*shape[:-1], 1, generator=gen, device="cuda"))).to(dtype)


def scales(*shape):
    return torch.full(shape, -7.0, device="cuda")


def codes(*shape):
    return torch.full(shape, 9, dtype=U8, device="cuda")


def rows_valid(kind, m, rng):
    """(arguments, slots, flags of valid rows [slots * m])"""
    if kind == "dense":
        return {}, 1, np.ones(m, bool)
    if kind == "contiguous":
        counts = rng.multinomial(max(0, m - 128 * 5), [0.1, 0.5, 0.0, 0.4])
        layout, _ = ref.contiguous_layout(counts, m)
        # a block of padding between the experts and a hole in a block
        layout[rng.integers(0, m)] = -1
        return dict(grouped_layout=torch.from_numpy(layout).cuda()), 1, layout >= 0
    counts = rng.integers(0, m + 1, 5)
    counts[0], counts[1], counts[2] = 0, m, -3
    given = counts.copy()
    given[1] = m + 7                           # clamped
    valid = np.arange(m)[None, :] < np.clip(counts, 0, m)[:, None]
    return dict(masked_m=torch.from_numpy(given.astype(np.int32)).cuda()), 5, valid.reshape(-1)


@pytest.mark.parametrize("kind,m,f", [("dense", 1, 128), ("dense", 33, 384), ("dense", 300, 2048),
                                      ("contiguous", 128, 256), ("contiguous", 1536, 640),
                                      ("masked", 1, 128), ("masked", 7, 256), ("masked", 64, 2048),
                                      ("masked", 150, 384)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_forward(gen, kind, m, f, act):
    print(f"[gpu] gated {kind} {m}x{f} {act}", flush=True)
    more, slots, valid = rows_valid(kind, m, np.random.default_rng(m))
    g = rand(gen, slots, m, 2 * f)
    g[0, 0, :128] = 0.0                        # a block of zeros
    g.view(-1, 2 * f)[torch.from_numpy(~valid).cuda()] = NAN
    ld = fp8bs.get_sfa_ld(m)
    hq, sfh, gq, sfg = codes(slots, m, f), scales(slots, f // 128, ld), codes(slots, m, 2 * f), scales(slots, 2 * f // 128, ld)
    if kind != "masked":
        g, hq, sfh, gq, sfg = (t[0] for t in (g, hq, sfh, gq, sfg))
    fp8bs.fp8bs_gated_quantize(g, hq, sfh, gq, sfg, activation=act, **more)
    v = host(g).reshape(-1, 2 * f)[valid]
    rows = lambda t: host(t).reshape(slots * m, -1)  # noqa: E731
    per_row = lambda t: np.swapaxes(host(t).reshape(slots, -1, ld), 1, 2)  # noqa: E731
    # the checkpoint: bit for bit
    code, scale = ref.quantise(v, -1)
    assert np.array_equal(rows(gq)[valid], code)
    assert np.array_equal(per_row(sfg)[:, :m].reshape(slots * m, -1)[valid], scale)
    value, _, tol, _ = ref.activation(v[:, :f].astype(np.float64), act)
    up = v[:, f:].astype(np.float64)
    sh = per_row(sfh)[:, :m].reshape(slots * m, -1)
    ref.check_quantised(rows(hq)[valid], sh[valid], value * up,
                        tol * np.abs(up) + E * np.abs(value * up), -1, "h")
    for q, s in ((hq, sfh), (gq, sfg)):        # what is not valid is left as it was
        assert np.all(rows(q)[~valid] == 9)
        s = per_row(s)
        assert np.all(s[:, :m].reshape(slots * m, -1)[~valid] == -7.0) and np.all(s[:, m:] == -7.0)
    # without the checkpoint the same
    h2, s2 = torch.full_like(hq, 9), torch.full_like(sfh, -7.0)
    fp8bs.fp8bs_gated_quantize(g, h2, s2, activation=act, **more)
    assert torch.equal(h2, hq) and torch.equal(s2, sfh)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gates_at_the_ends_of_the_range(act):
    f = 128
    gates = [0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 20.0, -20.0, 80.0, -80.0, 87.5, -87.5, 90.0, -90.0,
             103.0, -103.0, 150.0, -150.0, 1e4, -1e4, 1e15, -1e15, 1e30, -1e30, 3e38, -3e38]
    g = torch.ones(len(gates), 2 * f, dtype=BF16, device="cuda")
    g[:, :f] = torch.tensor(gates, device="cuda")[:, None].to(BF16)
    hq, sfh = codes(len(gates), f), scales(1, fp8bs.get_sfa_ld(len(gates)))
    fp8bs.fp8bs_gated_quantize(g, hq, sfh, activation=act)
    v = host(g).astype(np.float64)
    value, slope, tol, tol_s = ref.activation(v[:, :f], act)
    # (far out the 64-bit formula itself is 0 times infinity: act is v or 0 there, act' 1 or 0, and
    # neither is off at all)
    far = ~(np.isfinite(value) & np.isfinite(slope) & np.isfinite(tol_s)) | (np.abs(v[:, :f]) > 1e3)
    value, slope = np.where(far, np.maximum(v[:, :f], 0), value), np.where(far, v[:, :f] > 0, slope)
    tol, tol_s = np.where(far, 0.0, tol), np.where(far, 0.0, tol_s)
    ref.check_quantised(host(hq), ref.row_scales(sfh, len(gates)), value, tol, -1, act)
    dh = torch.ones(len(gates), f, dtype=BF16, device="cuda")
    d = torch.empty_like(g)
    fp8bs.fp8bs_gated_quantize_backward(g, dh, d=d, activation=act)
    got = host(d).astype(np.float64)
    assert np.isfinite(got).all()
    want, off = np.concatenate([slope, value], -1), np.concatenate([tol_s, tol], -1)
    assert np.all(np.abs(got - want) <= off + 2.0 ** -8 * (np.abs(want) + off) + 2.0 ** -133)


def test_infinities_and_nan_stay_in_their_blocks(gen):
    g = rand(gen, 6, 512)
    clean = g.clone()
    g[1, 3], g[2, 300], g[3, 7], g[4, 400] = NAN, NAN, float("inf"), -float("inf")
    hq, sfh, gq, sfg = codes(6, 256), scales(2, 8), codes(6, 512), scales(4, 8)
    fp8bs.fp8bs_gated_quantize(g, hq, sfh, gq, sfg)
    h2, s2, g2, t2 = codes(6, 256), scales(2, 8), codes(6, 512), scales(4, 8)
    fp8bs.fp8bs_gated_quantize(clean, h2, s2, g2, t2)
    for row, col in ((1, 3), (2, 300)):
        assert int(gq[row, col]) & 127 == 127 and int(hq[row, col % 256]) & 127 == 127
        other = torch.ones(512, dtype=torch.bool, device="cuda")
        other[col // 128 * 128:col // 128 * 128 + 128] = False
        assert torch.equal(gq[row][other], g2[row][other])
    # an infinity: its block's scale is infinite, the others' codes are zeros
    for row, col in ((3, 7), (4, 400)):
        assert float(sfg[col // 128, row]) == float("inf") and int(gq[row, col]) & 127 == 127
        block = slice(col // 128 * 128, col // 128 * 128 + 128)
        assert int((gq[row, block] & 127 == 0).sum()) == 127
    assert torch.equal(hq[[0, 5]], h2[[0, 5]]) and torch.equal(gq[[0, 5]], g2[[0, 5]])


def expected_gradients(v, dh, act):
    """64-bit gradients and h, and how far 32-bit ones may be off"""
    f = v.shape[1] // 2
    value, slope, tol_a, tol_s = ref.activation(v[:, :f], act)
    up = v[:, f:]
    d = np.concatenate([dh * up * slope, dh * value], -1)
    tol = np.concatenate([np.abs(dh * up) * tol_s, np.abs(dh) * tol_a], -1) + 2 * E * np.abs(d)
    h = value * up
    return d, tol, h, tol_a * np.abs(up) + E * np.abs(h)


BACK = [("dense", 1, 128), ("dense", 127, 384), ("dense", 128, 2048), ("dense", 400, 256),
        ("contiguous", 128, 128), ("contiguous", 1536, 640), ("contiguous", 2048, 256)]


@pytest.mark.parametrize("kind,m,f", BACK)
@pytest.mark.parametrize("act,kept", itertools.product(["silu", "gelu_tanh"], [True, False]))
def test_backward(gen, kind, m, f, act, kept):
    print(f"[gpu] gated backward {kind} {m}x{f} {act} {kept}", flush=True)
    more, _, valid = rows_valid(kind, m, np.random.default_rng(m + 1))
    bad = torch.from_numpy(~valid).cuda()
    g, dh = rand(gen, m, 2 * f), rand(gen, m, f, size=0.1)
    if kept:
        gq, sfg = fp8bs.quantize_1x128(g)
        v = ref.values_1x128(gq, sfg)
        v = (ref.VALUES[host(gq)].astype(np.float32) * np.repeat(ref.row_scales(sfg, m), 128, -1)).astype(np.float64)
        gq[bad] = 127                          # NaN where no token is
        sfg[:, :m][:, bad] = NAN
        args = dict(g=gq, sfg=sfg)
    else:
        v = host(g).astype(np.float64)
        g[bad] = NAN
        args = dict(g=g)
    dh64 = host(dh).astype(np.float64)
    dh[bad] = NAN
    padded = (m + 127) // 128 * 128
    ld = fp8bs.get_sfa_ld(m)
    out = dict(d=torch.full((m, 2 * f), 9.0, dtype=BF16, device="cuda"), dq=codes(m, 2 * f),
               sfd=scales(2 * f // 128, ld), dqt=codes(padded, 2 * f), sfdt=scales(padded // 128, 2 * f),
               hqt=codes(padded, f), sfht=scales(padded // 128, f))
    fp8bs.fp8bs_gated_quantize_backward(dh=dh, **args, **out, **more, activation=act)
    d, tol, h, tol_h = expected_gradients(v, dh64, act)
    got = host(out["d"]).astype(np.float64)
    assert np.all(np.abs(got - d)[valid] <= (tol + 2.0 ** -8 * (np.abs(d) + tol) + 1e-38)[valid])
    assert np.all(got[~valid] == 9.0)
    ref.check_quantised(host(out["dq"])[valid], ref.row_scales(out["sfd"], m)[valid], d[valid], tol[valid], -1, "dq")
    assert np.all(host(out["dq"])[~valid] == 9) and np.all(ref.row_scales(out["sfd"], m)[~valid] == -7.0)
    assert np.all(host(out["sfd"])[:, m:] == -7.0)
    # along tokens: zeros at rows without a token and behind the last
    for q, s, want, off in ((out["dqt"], out["sfdt"], d, tol), (out["hqt"], out["sfht"], h, tol_h)):
        full = np.zeros((2, padded, want.shape[1]))
        full[0, :m], full[1, :m] = np.where(valid[:, None], want, 0.0), np.where(valid[:, None], off, 0.0)
        ref.check_quantised(host(q), host(s), full[0], full[1], 0, "columns")
        held = np.zeros(padded, bool)
        held[:m] = valid
        assert np.all(host(q)[~held] == 0)
    # each output alone is the same
    for names in (("d",), ("dq", "sfd"), ("dqt", "sfdt"), ("hqt", "sfht"), ("dq", "sfd", "hqt", "sfht")):
        one = {n: torch.full_like(out[n], 9.0 if n == "d" else -7.0 if n.startswith("sf") else 9) for n in names}
        fp8bs.fp8bs_gated_quantize_backward(dh=dh, **args, **one, **more, activation=act)
        assert all(torch.equal(one[n], out[n]) for n in names), names
    # and with one workgroup a tile, as of many tiles
    try:
        fp8bs.set_num_cus(1)
        for names in (tuple(out), ("d",), ("dq", "sfd"), ("dqt", "sfdt"), ("hqt", "sfht")):
            one = {n: torch.full_like(out[n], 9.0 if n == "d" else -7.0 if n.startswith("sf") else 9) for n in names}
            fp8bs.fp8bs_gated_quantize_backward(dh=dh, **args, **one, **more, activation=act)
            assert all(torch.equal(one[n], out[n]) for n in names), names
    finally:
        fp8bs.set_num_cus(0)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_are_the_formulas(act):
    """the reference's gradients against autograd and differences in 64 bits"""
    rng = np.random.default_rng(6)
    v, dh = rng.normal(size=(5, 16)) * 2, rng.normal(size=(5, 8))
    t = torch.from_numpy(v).requires_grad_()
    gate, up = t.chunk(2, -1)
    a = torch.nn.functional.silu(gate) if act == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
    (a * up * torch.from_numpy(dh)).sum().backward()
    d, _, h, _ = expected_gradients(v, dh, act)
    assert np.allclose(d, t.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(h, (a * up).detach().numpy(), rtol=1e-12, atol=1e-14)
    step = rng.normal(size=v.shape)
    at = lambda s: (expected_gradients(v + s * step, dh, act)[2] * dh).sum()  # noqa: E731
    assert abs((at(1e-5) - at(-1e-5)) / 2e-5 - (d * step).sum()) < 1e-7 * np.abs(d * step).sum()


COLUMNS = [(1, 128, False), (128, 128, False), (130, 384, False), (200, 416, False), (3, 16, False),
           (300, 2064, False), (127, 7168, False), (128, 256, True), (1536, 640, True),
           (2048, 1152, True)]


# (e4m3 rows have scales for 128 columns each)
@pytest.mark.parametrize("kind,m,n,grouped", [(kind, *c) for kind in ("e4m3", "bf16", "f32")
                                              for c in COLUMNS if kind != "e4m3" or c[1] % 128 == 0])
def test_columns(gen, kind, m, n, grouped):
    print(f"[gpu] columns {kind} {m}x{n} {grouped}", flush=True)
    more, _, valid = rows_valid("contiguous" if grouped else "dense", m, np.random.default_rng(n))
    bad = torch.from_numpy(~valid).cuda()
    x = rand(gen, m, n, dtype=F32 if kind == "f32" else BF16)
    x[:, 5] = 0.0                              # a column of zeros
    sfx = None
    if kind == "e4m3":
        x, sfx = fp8bs.quantize_1x128(x)
        v = (ref.VALUES[host(x)].astype(np.float32) * np.repeat(ref.row_scales(sfx, m), 128, -1)).astype(np.float32)
        x[bad] = 255
        sfx[:, :m][:, bad] = NAN
    else:
        v = host(x)
        x[bad] = NAN
    padded = (m + 127) // 128 * 128
    q, sf = codes(padded, n), scales(padded // 128, fp8bs.get_sfa_ld(n))
    fp8bs.fp8bs_quantize_128x1(x, q, sf, sfx, **more)
    full = np.zeros((padded, n), np.float32)
    full[:m] = np.where(valid[:, None], v, 0)
    code, scale = ref.quantise(full, 0)
    assert np.array_equal(host(q), code) and np.array_equal(host(sf), scale)
    q2, sf2 = fp8bs.quantize_128x1(x, sfx, **more)
    assert torch.equal(q2, q) and torch.equal(sf2, sf)


def test_columns_with_nan_and_infinity(gen):
    x = rand(gen, 256, 256, dtype=F32)
    x[3, 7], x[200, 9], x[4, 11] = NAN, float("inf"), -0.0
    q, sf = fp8bs.quantize_128x1(x)
    code, scale = ref.quantise(host(x), 0)
    assert ref.same_codes(host(q), code) and np.array_equal(host(sf), scale)
    assert np.isinf(host(sf)[1, 9]) and np.isfinite(host(sf)[0]).all()


def test_columns_feed_the_weight_gradient(gen):
    counts, m, n = [100, 0, 300, 1], 256, 384
    layout, ks = ref.contiguous_layout(counts)
    rows = len(layout)
    lay = torch.from_numpy(layout).cuda()
    a, b = rand(gen, rows, m), rand(gen, rows, n, size=0.1)
    a[lay < 0], b[lay < 0] = NAN, NAN
    aq, sfa = fp8bs.quantize_128x1(a, grouped_layout=lay)
    bq, sfb = fp8bs.quantize_128x1(b, grouped_layout=lay)
    d = torch.empty(len(counts), m, n, device="cuda")
    fp8bs.fp8bs_k_grouped_tn_contiguous(aq, sfa, bq, sfb, d, ks)
    # The product's own bound (tests/test_gpu_kgrouped.py): the matrix core keeps a chunk's sum of 128
    # products to 2^-8 of the largest of them; chunks are added in FP32.
    va, vb = ref.values_128x1(aq, sfa), ref.values_128x1(bq, sfb)
    at = 0
    for e, k in enumerate(ks):
        x, y = va[at:at + k], vb[at:at + k]
        size = np.abs(x).T @ np.abs(y)
        top = np.zeros((m, n))
        for c in range(0, k, 128):
            top += (np.abs(x[c:c + 128, :, None]) * np.abs(y[c:c + 128, None, :])).max(0)
        assert np.all(np.abs(host(d)[e] - x.T @ y) <= 2.0 ** -8 * top + (k / 128 + 5) * E * size)
        at += k


def test_the_cap_changes_no_result(gen):
    g, dh = rand(gen, 1024, 1024), rand(gen, 1024, 512)
    runs = []
    try:
        for cap in (0, 1, 30):
            fp8bs.set_num_cus(cap)
            hq, sfh, gq, sfg = codes(1024, 512), scales(4, 1024), codes(1024, 1024), scales(8, 1024)
            fp8bs.fp8bs_gated_quantize(g, hq, sfh, gq, sfg)
            out = dict(dq=codes(1024, 1024), sfd=scales(8, 1024), dqt=codes(1024, 1024),
                       sfdt=scales(8, 1024), hqt=codes(1024, 512), sfht=scales(8, 512))
            fp8bs.fp8bs_gated_quantize_backward(gq, dh, sfg, **out)
            runs.append((hq, sfh, gq, sfg, *out.values(), *fp8bs.quantize_128x1(gq, sfg)))
    finally:
        fp8bs.set_num_cus(0)
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_rows_past_4_gib(gen):
    m, f = 300032, 8192
    tail = rand(gen, 128, 2 * f)
    g = torch.zeros(m, 2 * f, dtype=BF16, device="cuda")
    g[-128:] = tail
    ld = fp8bs.get_sfa_ld(m)
    hq, sfh = torch.zeros(m, f, dtype=U8, device="cuda"), torch.zeros(f // 128, ld, device="cuda")
    gq, sfg = torch.zeros(m, 2 * f, dtype=U8, device="cuda"), torch.zeros(2 * f // 128, ld, device="cuda")
    fp8bs.fp8bs_gated_quantize(g, hq, sfh, gq, sfg)
    del g
    h1, s1, g1, t1 = codes(128, f), scales(f // 128, 128), codes(128, 2 * f), scales(2 * f // 128, 128)
    fp8bs.fp8bs_gated_quantize(tail, h1, s1, g1, t1)
    assert torch.equal(hq[-128:], h1) and torch.equal(gq[-128:], g1)
    assert torch.equal(sfh[:, m - 128:m], s1) and torch.equal(sfg[:, m - 128:m], t1)
    dh = torch.zeros(m, f, dtype=BF16, device="cuda")
    dh[-128:] = rand(gen, 128, f)
    dq, sfd = torch.zeros_like(gq), torch.zeros_like(sfg)
    dqt, sfdt = torch.zeros_like(gq), torch.zeros(m // 128, 2 * f, device="cuda")
    fp8bs.fp8bs_gated_quantize_backward(gq, dh, sfg, dq=dq, sfd=sfd, dqt=dqt, sfdt=sfdt)
    q1, r1, c1, k1 = codes(128, 2 * f), scales(2 * f // 128, 128), codes(128, 2 * f), scales(1, 2 * f)
    fp8bs.fp8bs_gated_quantize_backward(g1, dh[-128:].contiguous(), t1, dq=q1, sfd=r1, dqt=c1, sfdt=k1)
    assert torch.equal(dq[-128:], q1) and torch.equal(dqt[-128:], c1)
    assert torch.equal(sfd[:, m - 128:m], r1) and torch.equal(sfdt[-1], k1[0])
    q, sf = fp8bs.quantize_128x1(gq, sfg)
    q2, sf2 = fp8bs.quantize_128x1(g1, t1)
    assert torch.equal(q[-128:], q2) and torch.equal(sf[-1], sf2[0])


def test_refusals_on_the_device(gen):
    g, dh = rand(gen, 128, 512), rand(gen, 128, 256)
    hq, sfh = codes(128, 256), scales(2, 128)
    gq, sfg = fp8bs.quantize_1x128(g)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize(g, hq, sfh, activation="relu")
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize(g, hq[:, :128], sfh)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize(g, hq, sfh[:1])
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize(g, hq, sfh, gq)
    with pytest.raises(TypeError):
        fp8bs.fp8bs_gated_quantize(g.float(), hq, sfh)
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.fp8bs_gated_quantize(rand(gen, 128, 320), codes(128, 160), scales(1, 128))
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.fp8bs_gated_quantize(g[:100], hq[:100], scales(2, 100),
                                   grouped_layout=torch.zeros(100, dtype=I32, device="cuda"))
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize_backward(gq, dh, d=g)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize_backward(gq, dh, sfg)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize_backward(g, dh, sfg, d=g)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_quantize_backward(g, dh[:, :128], d=g)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_quantize_128x1(gq, gq, scales(1, 512))
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.quantize_128x1(rand(gen, 4, 24))
    with pytest.raises(ValueError):
        fp8bs.fp8bs_quantize_128x1(g[:100], codes(100, 512), scales(1, 512))
