"""The operators between the FP8 products at sizes whose inputs and outputs pass the caches by: the
same bits as from calls on parts of the rows, which the tests of each operator check (`-m gpu`).
Every operator works row by row, or by 128 rows, so the parts' results are the whole's."""
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture()
def gen():
    return torch.Generator(device="cuda").manual_seed(20)


def rand(gen, *shape, dtype=BF16):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def ld(n):
    return (n + 3) // 4 * 4


def codes(rows, n):
    return torch.full((rows, n), 0x55, dtype=torch.uint8, device="cuda")


def scales(groups, n):
    return torch.full((groups, ld(n)), -7.0, device="cuda")


def row_scales(sf, groups, rows):
    return sf.view(groups, ld(rows))[:, :rows]


def same(a, b):
    ints = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(ints), b.contiguous().view(ints))


@pytest.mark.parametrize("xt", [BF16, F32])
def test_norm(gen, xt):
    m, k, part = 9001, 4096, 1000
    x, res, w = rand(gen, m, k, dtype=xt), rand(gen, m, k), rand(gen, k)

    def run(x, res):
        n = len(x)
        y, s, q, sf, rstd = torch.empty_like(x), torch.empty_like(res), codes(n, k), scales(k // 128, n), torch.empty(n, device="cuda")
        fp8bs.fp8bs_rms_norm(x, w, res, s, y, q, sf, rstd)
        return y, s, q, rstd, row_scales(sf, k // 128, n).T
    whole = run(x, res)
    for r in range(0, m, part):
        for a, b in zip(whole, run(x[r:r + part], res[r:r + part])):
            assert same(a[r:r + part], b)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("keep", [False, True])
def test_gated(gen, act, keep):
    m, f, part = 15000, 1152, 1024
    g = rand(gen, m, 2 * f)

    def run(g):
        n = len(g)
        hq, sfh = codes(n, f), scales(f // 128, n)
        gq, sfg = (codes(n, 2 * f), scales(f // 64, n)) if keep else (None, None)
        fp8bs.fp8bs_gated_quantize(g, hq, sfh, gq, sfg, activation=act)
        out = [hq, row_scales(sfh, f // 128, n).T]
        return out + ([gq, row_scales(sfg, f // 64, n).T] if keep else [])
    whole = run(g)
    for r in range(0, m, part):
        for a, b in zip(whole, run(g[r:r + part])):
            assert same(a[r:r + part], b)


@pytest.mark.parametrize("kept", [False, True])
def test_gated_backward(gen, kept):
    m, f, part = 13000, 1152, 1024
    g, dh, sfg = rand(gen, m, 2 * f), rand(gen, m, f), None
    if kept:
        hq, sfh, gq, sfg = codes(m, f), scales(f // 128, m), codes(m, 2 * f), scales(f // 64, m)
        fp8bs.fp8bs_gated_quantize(g, hq, sfh, gq, sfg)
        g, sfg = gq, row_scales(sfg, f // 64, m)

    def run(g, dh, sfg):
        n = len(g)
        pad = (n + 127) // 128 * 128
        if sfg is not None:
            own = scales(f // 64, n)
            own[:, :n] = sfg
            sfg = own
        d, dq, sfd = torch.empty(n, 2 * f, dtype=BF16, device="cuda"), codes(n, 2 * f), scales(f // 64, n)
        dqt, sfdt, hqt, sfht = codes(pad, 2 * f), scales(pad // 128, 2 * f), codes(pad, f), scales(pad // 128, f)
        fp8bs.fp8bs_gated_quantize_backward(g, dh, sfg, d, dq, sfd, dqt, sfdt, hqt, sfht)
        return (d, dq, row_scales(sfd, f // 64, n).T, dqt, hqt), (sfdt, sfht)
    whole, blocks = run(g, dh, sfg)
    for r in range(0, m, part):
        got, own = run(g[r:r + part], dh[r:r + part], None if sfg is None else sfg[:, r:r + part])
        for a, b in zip(whole, got):
            assert same(a[r:r + len(b)], b)
        for a, b in zip(blocks, own):
            assert same(a[r // 128:r // 128 + len(b)], b)


@pytest.mark.parametrize("kind", ["e4m3", BF16, F32])
def test_columns(gen, kind):
    m, n, part = 12345, 4096, 1024
    x, sfx = rand(gen, m, n, dtype=F32 if kind is F32 else BF16), None
    if kind == "e4m3":
        x, sfx = fp8bs.quantize_1x128(x)
        sfx = row_scales(sfx, n // 128, m)

    def run(x, sfx):
        if sfx is not None:
            own = scales(n // 128, len(x))
            own[:, :len(x)] = sfx
            sfx = own
        return fp8bs.quantize_128x1(x, sfx)
    q, sf = run(x, sfx)
    for r in range(0, m, part):
        a, b = run(x[r:r + part], None if sfx is None else sfx[:, r:r + part])
        assert same(q[r:r + len(a)], a) and same(sf[r // 128:r // 128 + len(b)], b)


@pytest.mark.parametrize("t", [BF16, F32])
def test_dispatch_and_combine(gen, t):
    tokens, topk, g, k, part = 5000, 3, 8, 4096, 500
    ids = torch.randint(-1, g, (tokens, topk), generator=gen, device="cuda")
    x, sfx = fp8bs.quantize_1x128(rand(gen, tokens, k))
    out = fp8bs.moe_dispatch(ids, x, g, sfx)
    pos, m = out.positions.long(), len(out.a)
    sf, sfx = row_scales(out.sfa, k // 128, m), row_scales(sfx, k // 128, tokens)
    for j in range(topk):
        there = pos[:, j] >= 0
        assert same(out.a.view(torch.uint8)[pos[there, j]], x.view(torch.uint8)[there])
        assert same(sf[:, pos[there, j]], sfx[:, there])
    d, w, dy = rand(gen, m, k), torch.rand(tokens, topk, generator=gen, device="cuda"), rand(gen, tokens, k, dtype=t)

    def forward(lo, hi):
        y = torch.empty(hi - lo, k, dtype=t, device="cuda")
        fp8bs.fp8bs_moe_combine(d, out.positions[lo:hi], y, w[lo:hi])
        return y

    def back(lo, hi, outs):
        dw = torch.empty(hi - lo, topk, device="cuda")
        fp8bs.fp8bs_moe_combine_backward(dy[lo:hi], out.positions[lo:hi], d, w[lo:hi], *outs, dweights=dw)
        return dw
    new = lambda: (torch.full((m, k), 3.0, dtype=BF16, device="cuda"), codes(m, k), scales(k // 128, m))
    y, outs, parts = forward(0, tokens), new(), new()
    dw = back(0, tokens, outs)
    for lo in range(0, tokens, part):
        assert same(y[lo:lo + part], forward(lo, lo + part))
        assert same(dw[lo:lo + part], back(lo, lo + part, parts))
    for a, b in zip(outs, parts):
        assert same(a, b)
