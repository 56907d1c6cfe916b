"""GPU tests of the operators together, as a mixture-of-experts layer uses them: a training step
(norm, dispatch, gate and up projections, gated activation, down projection, combine, and the whole
way back to the inputs' and weights' gradients) and a decode step in a captured graph.

The training step is compared with autograd in 64 bits on the same bf16 inputs and weights.  What
separates the two are the roundings to e4m3, each at most 2^-4 of a value (2^-4 of a block's norm):
relative errors of a product's factors add.  Forward: the normed row, both weights and the activation,
4 roundings; every gradient passes at most 4 more on its way and back (the outgoing gradient, dgate
and dup, a weight, an operand along tokens), and the checkpoint's, through which the activation is
looked at again, 2: relative error of a norm at most 4 x 2^-4 and 10 x 2^-4, if no rounding averaged
out.  (A transposed, shifted or missing operand gives an error above 1.)"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture
def gen():
    return torch.Generator("cuda").manual_seed(41)


def scales(*shape):
    return torch.empty(shape, device="cuda")


def codes(*shape):
    return torch.empty(shape, dtype=U8, device="cuda")


def weights(gen, g, rows, k):
    return (torch.randn(g, rows, k, generator=gen, device="cuda") / k ** 0.5).to(BF16)


def train_step(x, res, nw, ids, rw, w13, w2, dy, dres):
    """one layer forward and back: y, residual, and the gradients of x, nw, rw, w13 and w2"""
    tokens, k = x.shape
    g, f = w13.shape[0], w2.shape[2]
    q13, s13 = fp8bs.quantize_128x128(w13)
    q2, s2 = fp8bs.quantize_128x128(w2)
    # the transposed weights, for the gradients of the products' inputs
    t13, st13 = fp8bs.quantize_128x128(w13.transpose(1, 2).contiguous())
    t2, st2 = fp8bs.quantize_128x128(w2.transpose(1, 2).contiguous())
    # forward
    xq, sx, s, rstd = fp8bs.rms_norm_1x128(x, nw, res)
    a = fp8bs.moe_dispatch(ids, xq, g, sx)
    m = a.a.shape[0]
    lay = a.group_data
    gate_up = torch.empty(m, 2 * f, dtype=BF16, device="cuda")
    fp8bs.fp8bs_grouped_contiguous_nt(a.a, a.sfa, q13, s13, gate_up, lay)
    hq, sh, kq, sk = codes(m, f), scales(f // 128, m), codes(m, 2 * f), scales(2 * f // 128, m)
    fp8bs.fp8bs_gated_quantize(gate_up, hq, sh, kq, sk, grouped_layout=lay)
    d = torch.empty(m, k, dtype=BF16, device="cuda")
    fp8bs.fp8bs_grouped_contiguous_nt(hq, sh, q2, s2, d, lay)
    y = torch.empty(tokens, k, device="cuda")
    fp8bs.fp8bs_moe_combine(d, a.positions, y, rw)
    # back
    ddq, sdd, drw = codes(m, k), scales(k // 128, m), torch.empty_like(rw)
    fp8bs.fp8bs_moe_combine_backward(dy, a.positions, d, rw, q=ddq, sfa=sdd, dweights=drw)
    dh = torch.empty(m, f, dtype=BF16, device="cuda")
    fp8bs.fp8bs_grouped_contiguous_nt(ddq, sdd, t2, st2, dh, lay)
    dq, sd = codes(m, 2 * f), scales(2 * f // 128, m)
    dqt, sdt, hqt, sht = codes(m, 2 * f), scales(m // 128, 2 * f), codes(m, f), scales(m // 128, f)
    fp8bs.fp8bs_gated_quantize_backward(kq, dh, sk, dq=dq, sfd=sd, dqt=dqt, sfdt=sdt, hqt=hqt, sfht=sht,
                                        grouped_layout=lay)
    da = torch.empty(m, k, dtype=BF16, device="cuda")
    fp8bs.fp8bs_grouped_contiguous_nt(dq, sd, t13, st13, da, lay)
    dxn = torch.empty(tokens, k, device="cuda")
    fp8bs.fp8bs_moe_combine(da, a.positions, dxn)
    dx, dnw = torch.empty_like(s), torch.empty(k, device="cuda")
    fp8bs.fp8bs_rms_norm_backward(s, rstd, nw, dxn, dx, dres, dnw)
    # weight gradients: operands along tokens, groups of the experts' padded counts
    ks = [(c + 127) // 128 * 128 for c in a.counts.tolist()]
    rows = sum(ks)
    ddt, sddt = fp8bs.quantize_128x1(ddq, sdd, lay)
    at, sat = fp8bs.quantize_128x1(a.a, a.sfa, lay)
    dw13, dw2 = torch.empty(w13.shape, device="cuda"), torch.empty(w2.shape, device="cuda")
    cut = lambda q, sf: (q[:rows], sf[:rows // 128])  # noqa: E731
    fp8bs.fp8bs_k_grouped_tn_contiguous(*cut(dqt, sdt), *cut(at, sat), dw13, ks)
    fp8bs.fp8bs_k_grouped_tn_contiguous(*cut(ddt, sddt), *cut(hqt, sht), dw2, ks)
    return y, s, dict(x=dx, nw=dnw, rw=drw, w13=dw13, w2=dw2)


def in_64_bits(x, res, nw, ids, rw, w13, w2, dy, dres):
    x, res, nw, rw, w13, w2 = (t.double().requires_grad_() for t in (x, res, nw, rw, w13, w2))
    s = x + res
    n = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * nw
    y = torch.zeros_like(s)
    f = w2.shape[2]
    for e in range(w13.shape[0]):
        for j in range(ids.shape[1]):
            t = torch.nonzero(ids[:, j] == e)[:, 0]
            h = n[t] @ w13[e].t()
            out = (torch.nn.functional.silu(h[:, :f]) * h[:, f:]) @ w2[e].t()
            y = y.index_add(0, t, out * rw[t, j, None])
    ((y * dy.double()).sum() + (s * dres.double()).sum()).backward()
    return y.detach(), dict(x=x.grad, nw=nw.grad, rw=rw.grad, w13=w13.grad, w2=w2.grad)


def inputs(gen, tokens, topk, g, k, f, lost):
    x, res = (torch.randn(tokens, k, generator=gen, device="cuda").to(BF16) for _ in range(2))
    nw = 1 + 0.1 * torch.randn(k, generator=gen, device="cuda")
    ids = torch.rand(tokens, g + lost, generator=gen, device="cuda").topk(topk).indices
    ids[ids >= g] = -1
    ids[ids == 1] = 0                          # an expert without tokens, one chosen twice
    rw = torch.rand(tokens, topk, generator=gen, device="cuda")
    dy = torch.randn(tokens, k, generator=gen, device="cuda").to(BF16)
    dres = torch.randn(tokens, k, generator=gen, device="cuda").to(BF16)
    return x, res, nw, ids, rw, weights(gen, g, 2 * f, k), weights(gen, g, k, f), dy, dres


@pytest.mark.parametrize("tokens,topk,g,k,f,lost", [(300, 2, 4, 256, 128, 0), (77, 3, 8, 512, 384, 4),
                                                    (1500, 2, 4, 384, 256, 1)])
def test_training_step(gen, tokens, topk, g, k, f, lost):
    print(f"[gpu] training step {tokens}x{topk} of {g}, {k}, {f}", flush=True)
    args = inputs(gen, tokens, topk, g, k, f, lost)
    y, s, grads = train_step(*args)
    want, want_grads = in_64_bits(*args)
    assert torch.equal(s, (args[0].float() + args[1].float()).to(BF16))
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    errors = {n: rel(grads[n], want_grads[n]) for n in grads}
    print("relative errors: y %.3f" % rel(y, want), {n: round(e, 3) for n, e in errors.items()}, flush=True)
    assert rel(y, want) <= 4 * 2.0 ** -4
    for n, e in errors.items():
        assert e <= 10 * 2.0 ** -4, n
    # experts without tokens get zeros, each step the same bits
    assert bool((grads["w13"][1] == 0).all()) and bool((grads["w2"][1] == 0).all())
    again = train_step(*args)
    assert torch.equal(again[0], y) and all(torch.equal(again[2][n], grads[n]) for n in grads)


def test_training_step_of_no_tokens_here(gen):
    """every choice is of an expert elsewhere"""
    x, res, nw, ids, rw, w13, w2, dy, dres = inputs(gen, 40, 2, 4, 256, 128, 0)
    ids = torch.full_like(ids, -1)
    y, s, grads = train_step(x, res, nw, ids, rw, w13, w2, dy, dres)
    assert bool((y == 0).all()) and torch.equal(grads["x"], dres)
    for n in ("nw", "rw", "w13", "w2"):
        assert bool((grads[n] == 0).all()), n


@pytest.mark.parametrize("tokens", [1, 16, 300])
def test_decode_step_in_a_graph(gen, tokens):
    """norm, masked dispatch, both products, gated activation and combine, captured once; replays
    with new tokens and choices against the same calls made eagerly, and against 64 bits"""
    topk, g, k, f, slots = 2, 6, 512, 256, max(8, tokens)
    x, res, nw, ids, rw, w13, w2, _, _ = inputs(gen, tokens, topk, g, k, f, 2)
    q13, s13 = fp8bs.quantize_128x128(w13)
    q2, s2 = fp8bs.quantize_128x128(w2)
    ld, tl = fp8bs.get_sfa_ld(slots), fp8bs.get_sfa_ld(tokens)
    b = dict(out=torch.empty_like(res), q=codes(tokens, k), sq=scales(k // 128, tl), a=codes(g, slots, k),
             sa=scales(g, k // 128, ld), mm=torch.empty(g, dtype=I32, device="cuda"),
             pos=torch.empty(tokens, topk, dtype=I32, device="cuda"),
             counts=torch.empty(g, dtype=I32, device="cuda"),
             gu=torch.empty(g, slots, 2 * f, dtype=BF16, device="cuda"), hq=codes(g, slots, f),
             sh=scales(g, f // 128, ld), d=torch.empty(g, slots, k, dtype=BF16, device="cuda"),
             y=torch.empty(tokens, k, dtype=BF16, device="cuda"))

    def step():
        fp8bs.fp8bs_rms_norm(x, nw, res, b["out"], q=b["q"], sfa=b["sq"])
        fp8bs.fp8bs_moe_dispatch(ids, b["q"], b["a"], b["mm"], b["pos"], b["counts"], b["sq"], b["sa"])
        fp8bs.fp8bs_grouped_masked_nt(b["a"], b["sa"], q13, s13, b["gu"], b["mm"], expected_m=4)
        fp8bs.fp8bs_gated_quantize(b["gu"], b["hq"], b["sh"], masked_m=b["mm"])
        fp8bs.fp8bs_grouped_masked_nt(b["hq"], b["sh"], q2, s2, b["d"], b["mm"], expected_m=4)
        fp8bs.fp8bs_moe_combine(b["d"], b["pos"], b["y"], rw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        new = inputs(gen, tokens, topk, g, k, f, 2)
        x.copy_(new[0]), res.copy_(new[1]), ids.copy_(new[3]), rw.copy_(new[4])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in ("out", "y", "pos", "mm")}
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], b[n]) for n in got), turn
        want, _ = in_64_bits(x, res, nw, ids, rw, w13, w2, torch.zeros_like(x), torch.zeros_like(x))
        if float(want.norm()) > 0:
            assert float((got["y"].double() - want).norm() / want.norm()) <= 4 * 2.0 ** -4, turn


@pytest.mark.parametrize("tokens,in_place", [(40, False), (40, True), (500, False), (500, True)])
def test_way_back_in_a_graph(gen, tokens, in_place):
    """the gradients' operators (few rows and many, workspaces from the graph's own memory), captured once; replays
    with new inputs against the same calls made eagerly"""
    topk, g, k, f = 2, 4, 384, 128
    m = fp8bs.moe_capacity(tokens, topk, g)
    x, res, nw, ids, rw, _, _, dy, dres = inputs(gen, tokens, topk, g, k, f, 1)
    gate_up, d = (torch.randn(m, n, generator=gen, device="cuda").to(BF16) for n in (2 * f, k))
    rstd = torch.rand(tokens, generator=gen, device="cuda")
    kq, sk = fp8bs.quantize_1x128(gate_up)
    b = dict(ddq=codes(m, k), sdd=scales(k // 128, m), drw=torch.empty_like(rw), dq=codes(m, 2 * f), sd=scales(2 * f // 128, m),
             dqt=codes(m, 2 * f), sdt=scales(m // 128, 2 * f), hqt=codes(m, f), sht=scales(m // 128, f), ddt=codes(m, k),
             sddt=scales(m // 128, k), dxn=torch.empty(tokens, k, dtype=BF16, device="cuda"), dx=torch.empty_like(x),
             dnw=torch.empty(k, device="cuda"), positions=torch.empty(tokens, topk, dtype=I32, device="cuda"),
             lay=torch.empty(m, dtype=I32, device="cuda"), counts=torch.empty(g, dtype=I32, device="cuda"),
             a=torch.zeros(m, k, dtype=BF16, device="cuda"))
    for t in b.values():
        t.view(U8).zero_()

    def step():
        fp8bs.fp8bs_moe_dispatch(ids, x, b["a"], b["lay"], b["positions"], b["counts"])
        fp8bs.fp8bs_moe_combine_backward(dy, b["positions"], d, rw, q=b["ddq"], sfa=b["sdd"], dweights=b["drw"])
        fp8bs.fp8bs_gated_quantize_backward(kq, d[:, :f].contiguous(), sk, dq=b["dq"], sfd=b["sd"], dqt=b["dqt"], sfdt=b["sdt"],
                                            hqt=b["hqt"], sfht=b["sht"], grouped_layout=b["lay"])
        fp8bs.fp8bs_quantize_128x1(b["ddq"], b["ddt"], b["sddt"], b["sdd"], b["lay"])
        fp8bs.fp8bs_moe_combine(d, b["positions"], b["dxn"])
        dx = b["dxn"] if in_place else b["dx"]
        fp8bs.fp8bs_rms_norm_backward(x, rstd, nw, b["dxn"], dx, dres, b["dnw"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        new = inputs(gen, tokens, topk, g, k, f, 1)
        x.copy_(new[0]), ids.copy_(new[3]), rw.copy_(new[4]), dy.copy_(new[7]), dres.copy_(new[8])
        d.normal_(generator=gen)
        for t in b.values():                                          # (rows of no choice are not written)
            t.view(U8).zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in b.items()}
        for t in b.values():
            t.view(U8).zero_()
        step()
        torch.cuda.synchronize()
        for n, t in b.items():
            assert torch.equal(got[n].view(U8), t.view(U8)), (turn, n)
        assert bool((got["dnw"] != 0).any()) and bool((got["dqt"] != 0).any())


def test_dispatched_rows_through_the_4_bit_layer(gen):
    """bf16 rows dispatched for the MXFP4 feed-forward layer, and brought back"""
    tokens, topk, g, k, f = 200, 2, 4, 256, 128
    x, _, _, ids, rw, w13, w2, _, _ = inputs(gen, tokens, topk, g, k, f, 1)
    q13, s13 = fp8bs.quantize_mxfp4(w13)
    q2, s2 = fp8bs.quantize_mxfp4(w2)
    a = fp8bs.moe_dispatch(ids, x, g)
    d = fp8bs.feed_forward_mxfp4(a.a, q13, s13, q2, s2, grouped_layout=a.group_data)
    y = torch.empty(tokens, k, device="cuda")
    fp8bs.fp8bs_moe_combine(d, a.positions, y, rw)
    want = torch.zeros(tokens, k, device="cuda")
    for e in range(g):
        rows = fp8bs.feed_forward_mxfp4(x, q13[e], s13[e], q2[e], s2[e]).float()
        want += rows * (rw * (ids == e)).sum(-1, keepdim=True)
    assert float((y - want).norm() / want.norm()) < 2.0 ** -7


def test_two_streams_at_once(gen):
    """two training steps' calls in flight together, workspaces of their own"""
    args = [inputs(gen, 400, 2, 4, 256, 128, 0) for _ in range(2)]
    want = [train_step(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(train_step(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y, s, grads in got[i]:
            assert torch.equal(y, want[i][0])
            assert all(torch.equal(grads[n], want[i][2][n]) for n in grads)
