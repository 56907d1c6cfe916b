"""GPU tests of dispatch and combine: layouts, rows and scales exactly as made by hand; the weighted
way back against 64 bits (a sum of topk products in 32 bits: topk + 1 roundings of E = 2^-24, then
the output's); its gradients bit for bit, where they are one product, and within the roundings of a
dot product of k terms -- chains of at most k / 256 + 16 terms a lane, 8 exchanges -- for the weights'."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs
import _layer_ref as ref
from _layer_ref import E, HALF, host

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture
def gen():
    return torch.Generator("cuda").manual_seed(21)


def router(rng, tokens, topk, groups, kind):
    """choices: of all experts here; mostly of experts elsewhere; all of one expert; the same expert
    several times a token"""
    if kind == "here":
        ids = rng.integers(0, groups, (tokens, topk))
    elif kind == "elsewhere":
        ids = rng.integers(-3, 4 * groups, (tokens, topk))
    elif kind == "one":
        ids = np.full((tokens, topk), groups - 1)
    else:
        ids = np.repeat(rng.integers(0, groups, (tokens, 1)), topk, 1)
    return ids


def rows_of(gen, tokens, k, kind):
    """x, its scales, and 64-bit integer images of rows and scales"""
    if kind == "e4m3":
        x = torch.randint(0, 256, (tokens, k), generator=gen, device="cuda", dtype=torch.int32).to(U8)
        sfx = torch.rand((k // 128, fp8bs.get_sfa_ld(tokens)), generator=gen, device="cuda")
        return x, sfx
    return torch.randn(tokens, k, generator=gen, device="cuda").to(BF16 if kind == "bf16" else F32), None


def check(ids, x, sfx, got, groups, m, masked, fill):
    positions, data, counts, token = ref.layout_of(ids, groups, m, masked)
    assert np.array_equal(host(got.positions), positions)
    assert np.array_equal(host(got.group_data), data)
    assert np.array_equal(host(got.counts), counts)
    k = x.shape[1]
    held = token >= 0
    a = got.a.reshape(-1, k).cpu()
    assert torch.equal(a[torch.from_numpy(held)], x.cpu()[torch.from_numpy(token[held])])
    assert bool((a[torch.from_numpy(~held)] == fill).all())
    if sfx is not None:
        slots = groups if masked else 1
        sf = host(got.sfa).reshape(slots, k // 128, -1)
        rows = np.swapaxes(sf[..., :m], 1, 2).reshape(-1, k // 128)
        want = host(sfx)[:, :x.shape[0]].T
        assert np.array_equal(rows[held], want[token[held]])
        assert np.all(rows[~held] == -7.0) and np.all(sf[..., m:] == -7.0)


def dispatch(ids, x, sfx, groups, m, masked, fill=9):
    lead = (groups, m) if masked else (m,)
    k = x.shape[1]
    a = torch.full((*lead, k), fill, dtype=x.dtype, device="cuda")
    sfa = None if sfx is None else torch.full((*lead[:-1], k // 128, fp8bs.get_sfa_ld(m)), -7.0, device="cuda")
    data = torch.full((groups if masked else m,), 77, dtype=I32, device="cuda")
    positions = torch.full(ids.shape, 77, dtype=I32, device="cuda")
    counts = torch.full((groups,), 77, dtype=I32, device="cuda")
    fp8bs.fp8bs_moe_dispatch(ids, x, a, data, positions, counts, sfx, sfa)
    return fp8bs.Dispatched(a, sfa, data, positions, counts)


# one launch (few choices) and several (from 1024, with many groups 2048, on); rows of one piece, of
# several, longer than a workgroup's first pass; scales of up to more than 256 groups of columns
CASES = [
    # tokens, topk, groups, m (None: contiguous), k, type, kind
    (1, 1, 1, None, 128, "e4m3", "here"), (1, 8, 16, 4, 7168, "e4m3", "here"),
    (5, 2, 8, None, 640, "e4m3", "elsewhere"), (64, 8, 16, 64, 1280, "e4m3", "elsewhere"),
    (64, 8, 16, 20, 1280, "e4m3", "here"), (33, 3, 5, 7, 8, "bf16", "here"),
    (100, 8, 4, None, 24, "f32", "same"), (128, 8, 7, 100, 256, "e4m3", "one"),
    (127, 8, 200, None, 256, "bf16", "here"), (255, 8, 64, None, 256, "e4m3", "here"),
    (17, 2, 3, None, 33024, "e4m3", "here"), (9, 2, 3, 16, 33024, "e4m3", "here"),
    (9, 64, 1000, None, 128, "e4m3", "here"), (40, 1, 1024, 2, 128, "e4m3", "here"),
    (1000, 2, 8, None, 640, "e4m3", "here"), (1025, 1, 1, None, 128, "e4m3", "here"),
    (513, 4, 9, 250, 384, "e4m3", "elsewhere"), (700, 3, 5, 300, 1000, "bf16", "same"),
    (600, 7, 300, None, 256, "e4m3", "here"), (2048, 8, 64, None, 256, "e4m3", "one"),
    (5000, 8, 16, 3000, 128, "e4m3", "elsewhere"), (9000, 6, 1024, None, 128, "e4m3", "here"),
    (1100, 2, 4, None, 33024, "e4m3", "here"), (40000, 8, 3, None, 8, "f32", "here"),
    (2000, 1, 8, 0, 128, "e4m3", "here"), (20, 2, 8, 0, 128, "e4m3", "here"),
    # around the most choices of the one-launch kernels: 512, 2048 and, of 64 groups or more, 4096
    (171, 3, 8, None, 1152, "e4m3", "one"), (256, 8, 7, 2000, 256, "e4m3", "one"), (32, 64, 20, None, 264, "bf16", "here"),
    (683, 3, 63, None, 128, "e4m3", "elsewhere"), (512, 8, 64, None, 256, "e4m3", "one"), (1365, 3, 300, 16, 128, "e4m3", "elsewhere"),
    (4096, 1, 1024, None, 8, "f32", "same"), (4097, 1, 64, None, 8, "f32", "here"), (2049, 1, 3, None, 8, "bf16", "one"),
]


@pytest.mark.parametrize("tokens,topk,groups,m,k,kind,choices", CASES)
def test_dispatch(gen, tokens, topk, groups, m, k, kind, choices):
    print(f"[gpu] dispatch {tokens}x{topk} of {groups}, {m} rows of {k} {kind} {choices}", flush=True)
    rng = np.random.default_rng(tokens * 100 + topk)
    ids = router(rng, tokens, topk, groups, choices)
    x, sfx = rows_of(gen, tokens, k, kind)
    masked = m is not None
    m = fp8bs.moe_capacity(tokens, topk, groups) + 128 * (tokens % 2) if not masked else m
    for dtype in (torch.int32, torch.int64):
        got = dispatch(torch.from_numpy(ids).to(dtype).cuda(), x, sfx, groups, m, masked)
        check(ids, x, sfx, got, groups, m, masked, 9)


def test_ids_that_do_not_fit_32_bits(gen):
    ids = torch.tensor([[0, 1 << 32], [-(1 << 40), 1], [(1 << 32) + 1, 1 << 62]], device="cuda")
    x, sfx = rows_of(gen, 3, 128, "e4m3")
    got = dispatch(ids, x, sfx, 2, 256, False)
    assert host(got.positions).tolist() == [[0, -1], [-1, 128], [-1, -1]]
    assert host(got.counts).tolist() == [1, 1]


def test_no_tokens(gen):
    ids = torch.empty(0, 4, dtype=I32, device="cuda")
    x = torch.empty(0, 256, dtype=BF16, device="cuda")
    got = fp8bs.moe_dispatch(ids, x, 3)
    assert got.a.shape == (0, 256) and host(got.counts).tolist() == [0, 0, 0]
    for m in (128, 5000 * 128):
        got = dispatch(ids, x, None, 300, m, False)
        assert bool((got.group_data == -1).all()) and bool((got.counts == 0).all())
    got = fp8bs.moe_dispatch(ids, x, 3, max_m=5)
    assert host(got.group_data).tolist() == [0, 0, 0]
    y = torch.empty(0, 256, dtype=BF16, device="cuda")
    fp8bs.fp8bs_moe_combine(got.a, got.positions, y)
    fp8bs.fp8bs_moe_combine_backward(y, got.positions, dd=got.a)


def test_the_contiguous_layout_feeds_the_product(gen):
    """rows made by the allocating form, through the grouped product, against the tokens' own"""
    tokens, topk, g, n, k = 300, 3, 6, 256, 512
    rng = np.random.default_rng(5)
    ids = torch.from_numpy(rng.integers(-1, g, (tokens, topk))).cuda()
    x, sfx = fp8bs.quantize_1x128(torch.randn(tokens, k, generator=gen, device="cuda"))
    w, sfw = fp8bs.quantize_128x128(torch.randn(g, n, k, generator=gen, device="cuda"))
    got = fp8bs.moe_dispatch(ids, x, g, sfx)
    d = torch.zeros(got.a.shape[0], n, dtype=BF16, device="cuda")
    fp8bs.fp8bs_grouped_contiguous_nt(got.a, got.sfa, w, sfw, d, got.group_data)
    slots = fp8bs.moe_dispatch(ids, x, g, sfx, max_m=200)
    dm = torch.zeros(g, 200, n, dtype=BF16, device="cuda")
    fp8bs.fp8bs_grouped_masked_nt(slots.a, slots.sfa, w, sfw, dm, slots.group_data)
    each = torch.zeros(g, tokens, n, dtype=BF16, device="cuda")
    for e in range(g):
        fp8bs.fp8bs_dense_nt(x, sfx, w[e], sfw[e], each[e])
    want = torch.zeros(tokens, n, device="cuda")
    for t, j in np.argwhere(host(ids) >= 0):
        want[t] += each[int(ids[t, j]), t].float()
    for rows, of in ((d, got), (dm, slots)):
        y = torch.empty(tokens, n, device="cuda")
        fp8bs.fp8bs_moe_combine(rows, of.positions, y)
        # (instances of the product differ in the last bit of bf16)
        assert float((y - want).norm() / want.norm()) < 2.0 ** -7


SIZES = [(1, 1, 8), (3, 2, 7168), (64, 8, 1000), (7, 64, 136), (513, 3, 512), (33, 5, 4104)]


@pytest.mark.parametrize("tokens,topk,k", SIZES)
@pytest.mark.parametrize("yt", [BF16, F32])
def test_combine(gen, tokens, topk, k, yt):
    rng = np.random.default_rng(tokens)
    slots, m = 3, tokens * topk
    positions = rng.permutation(slots * m)[:tokens * topk].astype(np.int32)
    positions[rng.random(positions.shape) < 0.2] = -1
    positions[rng.random(positions.shape) < 0.1] = slots * m + 5          # left out as well
    positions = positions.reshape(tokens, topk)
    d = torch.randn(slots, m, k, generator=gen, device="cuda").to(BF16)
    unused = np.ones(slots * m, bool)
    used = positions[(positions >= 0) & (positions < slots * m)]
    unused[used] = False
    d.view(-1, k)[torch.from_numpy(unused).cuda()] = float("nan")         # never read
    w = torch.randn(tokens, topk, generator=gen, device="cuda")
    p = torch.from_numpy(positions).cuda()
    for weights in (w, None):
        for rows in (d, d.view(-1, k)):
            y = torch.full((tokens, k), 9.0, dtype=yt, device="cuda")
            fp8bs.fp8bs_moe_combine(rows, p, y, weights)
            here = (positions >= 0) & (positions < slots * m)
            v = host(d).reshape(-1, k).astype(np.float64)[np.where(here, positions, used[:1] if len(used) else 0)]
            f = np.where(here, host(w) if weights is not None else 1.0, 0.0).astype(np.float64)
            v = np.where(here[..., None], v, 0.0) * f[..., None]
            want, size = v.sum(1), np.abs(v).sum(1)
            tol = (topk + 1) * E * size
            assert np.all(np.abs(host(y) - want) <= tol + HALF[yt] * (np.abs(want) + tol))


@pytest.mark.parametrize("tokens,topk,k,slots", [(1, 1, 128, 1), (3, 2, 7168, 1), (64, 8, 1280, 4),
                                                 (9, 63, 256, 2), (130, 3, 4224, 1), (33, 5, 2048, 3)])
@pytest.mark.parametrize("gt", [BF16, F32])
def test_combine_backward(gen, tokens, topk, k, slots, gt):
    rng = np.random.default_rng(tokens)
    m = (2 * tokens * topk + slots - 1) // slots
    positions = rng.permutation(slots * m)[:tokens * topk].astype(np.int32)
    positions[rng.random(positions.shape) < 0.2] = -1
    positions[rng.random(positions.shape) < 0.1] = slots * m + 5
    positions = positions.reshape(tokens, topk)
    here = (positions >= 0) & (positions < slots * m)
    p = torch.from_numpy(positions).cuda()
    dy = (torch.randn(tokens, k, generator=gen, device="cuda") * 0.1).to(gt)
    dy[0, :128] = 0.0                                                     # a block of zeros
    d = torch.randn(slots, m, k, generator=gen, device="cuda").to(BF16)
    flags = torch.ones(slots * m, dtype=torch.bool)
    flags[torch.from_numpy(positions[here].astype(np.int64))] = False
    d.view(-1, k)[flags.cuda()] = float("nan")
    w = torch.randn(tokens, topk, generator=gen, device="cuda")
    w[0, 0] = 0.0
    for weights in (w, None):
        dd = torch.full((slots, m, k), 9.0, dtype=BF16, device="cuda")
        q = torch.full((slots, m, k), 9, dtype=U8, device="cuda")
        sfa = torch.full((slots, k // 128, fp8bs.get_sfa_ld(m)), -7.0, device="cuda")
        dw = torch.full((tokens, topk), 9.0, device="cuda")
        fp8bs.fp8bs_moe_combine_backward(dy, p, d, weights, dd, q, sfa, dw)
        f = host(w) if weights is not None else np.ones((tokens, topk), np.float32)
        prod = (f[..., None] * host(dy)[:, None, :]).astype(np.float32)
        rows, at = prod[here], positions[here]
        flat = host(dd).reshape(-1, k)
        assert np.array_equal(flat[at], ref.bf16(rows))
        code, scale = ref.quantise(rows, -1) if len(rows) else (rows.astype(np.uint8), rows[:, ::128])
        got = np.swapaxes(host(sfa)[..., :m], 1, 2).reshape(-1, k // 128)
        assert np.array_equal(host(q).reshape(-1, k)[at], code) and np.array_equal(got[at], scale)
        rest = np.ones(slots * m, bool)
        rest[at] = False
        assert np.all(flat[rest] == 9.0) and np.all(host(q).reshape(-1, k)[rest] == 9)
        assert np.all(got[rest] == -7.0) and np.all(host(sfa)[..., m:] == -7.0)
        v = host(d).reshape(-1, k).astype(np.float64)
        terms = np.zeros((tokens, topk, k))
        for t, j in np.argwhere(here):
            terms[t, j] = host(dy)[t].astype(np.float64) * v[positions[t, j]]
        tol = (k / 256 + 16 + 12) * E * np.abs(terms).sum(-1)
        assert np.all(np.abs(host(dw) - terms.sum(-1)) <= tol)
        assert np.all(host(dw)[~here] == 0.0)
        # each output alone; a matrix instead of slots; d not needed for the others
        for only in ("dd", "q", "dweights"):
            one = dict(dd=torch.full_like(dd, 9.0)) if only == "dd" else dict(
                q=torch.full_like(q, 9), sfa=torch.full_like(sfa, -7.0)) if only == "q" else dict(
                d=d, dweights=torch.full_like(dw, 9.0))
            fp8bs.fp8bs_moe_combine_backward(dy, p, weights=weights, **one)
            for name, want in (("dd", dd), ("q", q), ("sfa", sfa), ("dweights", dw)):
                assert name not in one or torch.equal(one[name], want)


def test_gradients_by_differences(gen):
    """<dispatch(x), g> = <x, combine(g)>, and combine's gradients against differences, which are
    exact for a bilinear form up to the roundings"""
    rng = np.random.default_rng(8)
    tokens, topk, g, k = 50, 3, 7, 256
    ids = torch.from_numpy(rng.integers(-1, g, (tokens, topk))).cuda()
    x = torch.randn(tokens, k, generator=gen, device="cuda")
    a = fp8bs.moe_dispatch(ids, x, g)
    cot = torch.randn(a.a.shape, generator=gen, device="cuda").to(BF16)
    dx = torch.empty(tokens, k, device="cuda")
    fp8bs.fp8bs_moe_combine(cot, a.positions, dx)
    held = a.group_data >= 0
    left = (a.a[held].double() * cot[held].double()).sum()
    assert abs(float(left - (x.double() * dx.double()).sum())) < 1e-5 * float(
        (x.double() * dx.double()).abs().sum())
    d = torch.randn(a.a.shape, generator=gen, device="cuda").to(BF16)
    w = torch.randn(tokens, topk, generator=gen, device="cuda")
    dy = torch.randn(tokens, k, generator=gen, device="cuda")
    dd, dw = torch.zeros_like(d), torch.empty_like(w)
    fp8bs.fp8bs_moe_combine_backward(dy, a.positions, d, w, dd=dd, dweights=dw)

    def loss(d, w):
        y = torch.empty(tokens, k, device="cuda")
        fp8bs.fp8bs_moe_combine(d, a.positions, y, w)
        return float((y.double() * dy.double()).sum())
    step = torch.randn(w.shape, generator=gen, device="cuda")
    got = (loss(d, w + step) - loss(d, w - step)) / 2
    assert abs(got - float((dw.double() * step.double()).sum())) < 1e-4 * abs(loss(d, w)) + 1e-3
    other = torch.randn(d.shape, generator=gen, device="cuda").to(BF16)
    change = loss(other, w)                    # linear in d: the derivative along `other`
    along = (dd.double() * other.double())[held].sum()
    # (dd is rounded to bf16: 2^-8 of each term)
    assert abs(change - float(along)) < 2.0 ** -8 * float((dd.double() * other.double())[held].abs().sum())


def test_streams_and_a_workspace_of_the_callers(gen):
    ids = torch.randint(0, 8, (2000, 4), generator=gen, device="cuda")
    x, sfx = rows_of(gen, 2000, 256, "e4m3")
    want = fp8bs.moe_dispatch(ids, x, 8, sfx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    m = fp8bs.moe_capacity(2000, 4, 8)
    ws = torch.full((fp8bs.moe_dispatch_workspace_size(fp8bs.LAYOUT_CONTIGUOUS, 2000, 4, 8, m),), 255,
                    dtype=U8, device="cuda")
    a, sfa = torch.empty_like(want.a), torch.empty_like(want.sfa)
    data, pos, counts = (torch.empty_like(t) for t in want[2:])
    torch.cuda.synchronize()
    fp8bs.fp8bs_moe_dispatch(ids, x, a, data, pos, counts, sfx, sfa, workspace=ws, stream=side)
    got = fp8bs.moe_dispatch(ids, x, 8, sfx, stream=side)
    side.synchronize()
    held = want.group_data >= 0
    for o in ((a, data, pos, counts), (got.a, got.group_data, got.positions, got.counts)):
        assert torch.equal(o[0][held], want.a[held])
        assert all(torch.equal(p, q) for p, q in zip(o[1:], want[2:]))
    with pytest.raises(fp8bs.FP8BSError):
        fp8bs.fp8bs_moe_dispatch(ids, x, a, data, pos, counts, sfx, sfa, workspace=ws[:64])


@pytest.mark.parametrize("tokens", [40, 3000])
def test_the_cap_changes_no_result(gen, tokens):
    ids = torch.randint(-2, 8, (tokens, 4), generator=gen, device="cuda")
    x, sfx = rows_of(gen, tokens, 1280, "e4m3")
    dy = torch.randn(tokens, 1280, generator=gen, device="cuda")
    w = torch.rand(tokens, 4, generator=gen, device="cuda")
    runs = []
    try:
        for cap in (0, 2, 33):
            fp8bs.set_num_cus(cap)
            got = dispatch(ids, x, sfx, 8, fp8bs.moe_capacity(tokens, 4, 8), False)
            d = got.a.to(BF16)
            q, sfa = torch.zeros_like(got.a), torch.zeros_like(got.sfa)
            dw, y = torch.empty_like(w), torch.empty_like(dy)
            fp8bs.fp8bs_moe_combine_backward(dy, got.positions, d, w, q=q, sfa=sfa, dweights=dw)
            fp8bs.fp8bs_moe_combine(d, got.positions, y, w)
            runs.append((*got, q, sfa, dw, y))
    finally:
        fp8bs.set_num_cus(0)
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("tokens", [30, 2000])
def test_captured_and_replayed(gen, tokens):
    g, k = 8, 512
    ids = torch.zeros(tokens, 2, dtype=I32, device="cuda")
    x, sfx = rows_of(gen, tokens, k, "e4m3")
    m = fp8bs.moe_capacity(tokens, 2, g)
    a, sfa = torch.zeros(m, k, dtype=U8, device="cuda"), torch.zeros(k // 128, m, device="cuda")
    data, counts = torch.zeros(m, dtype=I32, device="cuda"), torch.zeros(g, dtype=I32, device="cuda")
    pos = torch.zeros(tokens, 2, dtype=I32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fp8bs.fp8bs_moe_dispatch(ids, x, a, data, pos, counts, sfx, sfa)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8bs.fp8bs_moe_dispatch(ids, x, a, data, pos, counts, sfx, sfa)
    rng = np.random.default_rng(2)
    for turn in range(4):
        new = rng.integers(-1, g, (tokens, 2)).astype(np.int32)
        ids.copy_(torch.from_numpy(new))
        a.fill_(9)
        sfa.fill_(-7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(new, x, sfx, fp8bs.Dispatched(a, sfa, data, pos, counts), g, m, False, 9)


def test_rows_past_4_gib(gen):
    tokens, topk, k = 20000, 8, 32768
    ids = torch.arange(8, device="cuda", dtype=I32).repeat(tokens, 1)
    x, sfx = rows_of(gen, tokens, k, "e4m3")
    got = fp8bs.moe_dispatch(ids, x, 8, sfx)
    at = got.positions[-3:].reshape(-1).long()
    assert int(at.max()) * k > 1 << 32
    assert torch.equal(got.a[at].view(3, 8, k), x[-3:, None].expand(3, 8, k))
    assert torch.equal(got.sfa[:, at].view(-1, 3, 8), sfx[:, tokens - 3:tokens, None].expand(-1, 3, 8))
    d = got.a[:, :8192].to(BF16).contiguous()
    y = torch.empty(tokens, 8192, device="cuda")
    fp8bs.fp8bs_moe_combine(d, got.positions, y)
    assert torch.equal(y[-3:], 8.0 * x[-3:, :8192].float())
    dd = torch.zeros_like(d)
    fp8bs.fp8bs_moe_combine_backward(y, got.positions, dd=dd)
    assert torch.equal(dd[at].view(3, 8, -1), y[-3:, None].to(BF16).expand(3, 8, 8192))


def test_refusals_on_the_device(gen):
    ids = torch.zeros(4, 2, dtype=I32, device="cuda")
    x, sfx = rows_of(gen, 4, 256, "e4m3")
    m = fp8bs.moe_capacity(4, 2, 2)
    a, sfa = torch.zeros(m, 256, dtype=U8, device="cuda"), torch.zeros(2, m, device="cuda")
    data, pos = torch.zeros(m, dtype=I32, device="cuda"), torch.zeros_like(ids)
    counts = torch.zeros(2, dtype=I32, device="cuda")
    call = fp8bs.fp8bs_moe_dispatch
    with pytest.raises(TypeError):
        call(ids.float(), x, a, data, pos, counts, sfx, sfa)
    with pytest.raises(ValueError):
        call(ids[:3], x, a, data, pos[:3], counts, sfx, sfa)
    with pytest.raises(ValueError):
        call(ids, x, a, data, pos, counts, None, sfa)
    with pytest.raises(ValueError):
        call(ids, x, a, data, pos, counts, sfx, sfa[:1])
    with pytest.raises(TypeError):
        call(ids, x.float(), a, data, pos, counts)
    with pytest.raises(ValueError):
        call(ids, x.to(BF16), a.to(BF16), data, pos, counts, sfx, sfa)
    with pytest.raises(ValueError):
        call(ids, x, a, data[:5], pos, counts, sfx, sfa)
    with pytest.raises(fp8bs.FP8BSError):
        call(ids, x, a[:128], data[:128], pos, counts, sfx, torch.zeros(2, 128, device="cuda"))
    y = torch.zeros(4, 256, device="cuda")
    with pytest.raises(TypeError):
        fp8bs.fp8bs_moe_combine(a, pos, y)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_moe_combine(a.to(BF16), pos[:3], y)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_moe_combine_backward(y, pos, dweights=torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        fp8bs.fp8bs_moe_combine_backward(y, pos)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_moe_combine_backward(y, pos, q=a)
