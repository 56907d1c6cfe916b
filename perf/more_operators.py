"""What is measured of the operators between the products of an FP8 mixture-of-experts layer:
the root-mean-square norm with the residual's addition and e4m3 output, with its gradients; the
dispatch of tokens to their experts and the weighted way back, with its gradients; the gated
activation with e4m3 output and an e4m3 checkpoint, with the backward pass from the checkpoint;
and the quantiser along tokens for weight gradients.

Quantisation here: a block of 128 values shares a = max(largest magnitude, 1e-4); scale = a / 448
and code = e4m3(clamp(x * (448 / a), -448, 448)).  "1x128": 128 columns of a row, scales K-group-
major, f32 [k/128][ld], ld = rows rounded up to a multiple of 4.  "128x1": 128 rows of a column,
f32 [ceil(rows/128)][ld(n)]; rows are padded with zeros to a multiple of 128.

Norm: s = x + residual, y = s / sqrt(mean(s^2) + eps) * w.

Dispatch: assignment (t, j) -- token t's j-th choice, expert ids[t][j] -- goes behind the expert's
earlier assignments.  "contiguous": experts' segments one after another, each padded to a multiple
of 128 rows; "masked": a slot of max_m rows per expert, later assignments dropped.  Choices outside
0 .. g-1 (experts of another device) are dropped.  positions[t][j] is the row, -1 if dropped.
Combine: y[t] = sum_j w[t][j] d[positions[t][j]].

Gated activation: h = act(gate) * up, gate the columns 0 .. f-1, up f .. 2f-1.

Rows that hold no token are not written (along tokens: zeros); outputs' buffers start as zeros.
"""
import math

import torch

own = False

EPS = 1e-6


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token of a decode step before its experts: the smallest call, latency counts
        dict(name="norm 1x7168", op="norm", rows=1, k=7168, x="bf16", res="bf16"),
        # a prefill or training batch
        dict(name="norm 16384x7168", op="norm", rows=16384, k=7168, x="bf16", res="bf16"),
        # the training batch's gradients
        dict(name="norm backward 16384x7168", op="norm_backward", rows=16384, k=7168, dy="bf16",
             res="bf16"),
        # a decode step of 64 tokens, eight choices of 64 experts, 16 of them here
        dict(name="dispatch masked g16", op="dispatch", layout="masked", tokens=64, topk=8,
             experts=64, g=16, m=64, k=7168, x="e4m3"),
        # a training batch, two choices of eight experts
        dict(name="dispatch contiguous g8", op="dispatch", layout="contiguous", tokens=16384,
             topk=2, experts=8, g=8, k=7168, x="e4m3"),
        # the way back of the decode step
        dict(name="combine masked g16", op="combine", layout="masked", tokens=64, topk=8,
             experts=64, g=16, m=64, k=7168, y="bf16"),
        # the way back's gradients of the training batch
        dict(name="combine backward contiguous g8", op="combine_backward", layout="contiguous",
             tokens=16384, topk=2, experts=8, g=8, k=7168, dy="bf16", wide=False),
        # activation of a decode step over sixteen experts' slots
        dict(name="gated masked g16", op="gated", layout="masked", m=64, f=2048, g=16,
             act="silu", keep=False),
        # activation of a training batch over eight experts, kept for the backward pass
        dict(name="gated contiguous g8", op="gated", layout="contiguous", m=33280, f=2048, g=8,
             act="silu", keep=True),
        # its gradients from what was kept
        dict(name="gated backward contiguous g8", op="gated_backward", layout="contiguous",
             m=33280, f=2048, g=8, act="silu", x="e4m3"),
        # a small odd batch's gradient on its way to a weight gradient
        dict(name="columns 200x416", op="columns", layout="dense", m=200, n=416, g=1, x="bf16"),
        # a kept operand on its way to a weight gradient
        dict(name="columns contiguous g8", op="columns", layout="contiguous", m=33280, n=7168,
             g=8, x="e4m3"),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        """log-uniform over lo .. hi, a multiple of step"""
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(round(v / step)) * step)

    op = rng.choice(["norm", "norm_backward", "dispatch", "combine", "combine_backward", "gated",
                     "gated_backward", "columns"])
    types = ["bf16", "f32"]
    if op == "norm":
        return dict(op=op, rows=size(1, 12000), k=size(128, 7168, 128), x=rng.choice(types),
                    res=rng.choice(types))
    if op == "norm_backward":
        return dict(op=op, rows=size(1, 8000), k=size(128, 7168, 8), dy=rng.choice(types),
                    res=rng.choice(types))
    if op in ("dispatch", "combine", "combine_backward"):
        g = size(1, 64)
        c = dict(op=op, layout=rng.choice(["contiguous", "masked"]), topk=rng.randint(1, 8),
                 experts=g * rng.choice([1, 1, 2, 8]), g=g, k=size(128, 7168, 128))
        if c["layout"] == "masked":
            c.update(tokens=size(1, 512))
            # slots from too small for the fullest expert to ample
            c["m"] = max(1, int(c["tokens"] * c["topk"] / c["experts"] * rng.uniform(0.7, 3.0)))
        else:
            c.update(tokens=size(1, 24000 // c["topk"]))
        if op == "dispatch":
            c["x"] = rng.choice(["e4m3", "bf16"])
        elif op == "combine":
            c["y"] = rng.choice(types)
        else:
            c.update(dy=rng.choice(types), wide=rng.random() < 0.5)
        return c
    layouts = ["dense", "contiguous"] + (["masked"] if op == "gated" else [])
    c = dict(op=op, layout=rng.choice(layouts), g=1)
    if c["layout"] == "dense":
        c["m"] = size(1, 16384)
    elif c["layout"] == "contiguous":
        c.update(m=size(128, 24000, 128), g=size(1, 16))
    else:
        c.update(m=size(1, 512), g=size(1, 16))
    if op == "columns":
        c["x"] = rng.choice(["e4m3", "bf16", "f32"])
        c["n"] = size(128, 4096, 128) if c["x"] == "e4m3" else size(16, 4096, 16)
        return c
    c.update(f=size(128, 2048, 128), act=rng.choice(["silu", "gelu_tanh"]))
    if op == "gated":
        c["keep"] = rng.random() < 0.5
    else:
        c["x"] = rng.choice(["e4m3", "bf16"])
    return c


BYTES = {"bf16": 2, "f32": 4, "e4m3": 1 + 4 / 128}


def capacity(tokens, topk, g):
    """Rows that the contiguous layout can need."""
    n = tokens * topk
    return (n + 127 * min(g, n)) // 128 * 128


def work(case):
    op = case["op"]
    e4m3 = BYTES["e4m3"]
    if op == "norm":
        n = case["rows"] * case["k"]
        return {"bytes": n * (BYTES[case["x"]] + 2 * BYTES[case["res"]] + e4m3) + 2.0 * case["k"],
                "flops": 8.0 * n}
    if op == "norm_backward":
        n = case["rows"] * case["k"]
        return {"bytes": n * (BYTES[case["dy"]] + 3 * BYTES[case["res"]]) + 6.0 * case["k"],
                "flops": 12.0 * n}
    if op in ("dispatch", "combine", "combine_backward"):
        t, k, n = case["tokens"], case["k"], case["tokens"] * case["topk"]
        # assignments to an expert here that find a row, and tokens with one of them
        rows = n * case["g"] // case["experts"]
        if case["layout"] == "masked":
            rows = min(rows, case["g"] * case["m"])
        here = t * (1.0 - (1.0 - case["g"] / case["experts"]) ** case["topk"])
        if op == "dispatch":
            size = BYTES[case["x"]]
            return {"bytes": k * size * (here + rows) + 12.0 * n, "flops": float(n)}
        if op == "combine":
            return {"bytes": k * (2.0 * rows + BYTES[case["y"]] * t) + 8.0 * n,
                    "flops": 2.0 * rows * k}
        out = e4m3 + (2 if case["wide"] else 0)
        return {"bytes": k * (BYTES[case["dy"]] * here + rows * (2.0 + out)) + 12.0 * n,
                "flops": 6.0 * rows * k}
    # rows that hold a token, as prepare() fills them on average, and rows written along tokens
    rows, g = case["m"], case["g"]
    every = (rows + 127) // 128 * 128
    if case["layout"] == "contiguous":
        rows = max(1, case["m"] - 64 * min(g, case["m"] // 128))
    elif case["layout"] == "masked":
        rows = g * (case["m"] + 1) // 2
    if op == "columns":
        return {"bytes": case["n"] * (rows * BYTES[case["x"]] + every * e4m3),
                "flops": 3.0 * rows * case["n"]}
    f = case["f"]
    if op == "gated":
        return {"bytes": rows * f * (4.0 + e4m3 * (3 if case["keep"] else 1)),
                "flops": 12.0 * rows * f}
    return {"bytes": f * (rows * (2 * BYTES[case["x"]] + 2.0 + 2 * e4m3) + every * 3 * e4m3),
            "flops": 40.0 * rows * f}


# ---- inputs ----------------------------------------------------------------

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ld(rows):
    return (rows + 3) // 4 * 4


def _activations(shape, gen, dtype):
    """Hidden states: unit variance, tokens of different size, a few large channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    size = torch.exp(0.3 * torch.randn(shape[:-1], generator=gen, device="cuda"))
    channel = torch.where(torch.rand(shape[-1], generator=gen, device="cuda") < 0.01, 6.0, 1.0)
    return (x * size.unsqueeze(-1) * channel).to(dtype)


def _gradients(shape, gen, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * 0.05).to(dtype)


def _zeros(shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _scales(lead, rows, k):
    """1x128 scales of [*lead, rows, k]."""
    return _zeros((*lead, k // 128, _ld(rows)), torch.float32)


def _kept(x):
    """A kept operand: codes and 1x128 scales, made outside the measured calls."""
    code, scale = _rows_128(x.float())
    return code.view(torch.uint8), _major(scale)


def _rows(s, layout, m, g, seed):
    """Which rows hold a token."""
    host = torch.Generator().manual_seed(seed)
    if layout == "masked":
        s["masked_m"] = torch.randint(0, m + 1, (g,), generator=host).to(torch.int32).cuda()
        s["valid"] = torch.arange(m, device="cuda")[None, :] < s["masked_m"][:, None]
    elif layout == "contiguous":
        # cut the 128-row blocks at random places into one run per expert (empty ones too);
        # the last block of a run ends in up to 127 rows of padding
        blocks = m // 128
        cuts = torch.randint(0, blocks + 1, (g - 1,), generator=host).sort().values.tolist()
        at = [128 * b for b in [0] + cuts + [blocks]]
        pad = torch.randint(0, 128, (g,), generator=host).tolist()
        index = torch.full((m,), -1, dtype=torch.int32)
        for e, (a, b, p) in enumerate(zip(at[:-1], at[1:], pad)):
            index[a:(b - p if b > a else b)] = e
        s["grouped_layout"] = index.cuda()
        s["valid"] = s["grouped_layout"] >= 0
    else:
        s["valid"] = torch.ones(m, dtype=torch.bool, device="cuda")


def _router(case, gen):
    """ids int32 [tokens][topk], weights f32: distinct experts per token, some more popular."""
    score = torch.randn(case["tokens"], case["experts"], generator=gen, device="cuda")
    score = score + 0.5 * torch.randn(case["experts"], generator=gen, device="cuda")
    topk = min(case["topk"], case["experts"])
    top = torch.topk(score, topk, dim=-1)
    weights = torch.exp(top.values - top.values[:, :1])
    weights = weights / weights.sum(-1, keepdim=True)
    if topk < case["topk"]:                     # fewer experts than choices: the rest unused
        more = (0, case["topk"] - topk)
        return (torch.nn.functional.pad(top.indices, more, value=-1).to(torch.int32),
                torch.nn.functional.pad(weights, more))
    return top.indices.to(torch.int32).contiguous(), weights.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(op=op)
    if op in ("norm", "norm_backward"):
        rows, k = case["rows"], case["k"]
        res = DTYPES[case["res"]]
        s["weight"] = (1.0 + 0.1 * torch.randn(k, generator=gen, device="cuda")).to(torch.bfloat16)
        s["s"] = _activations((rows, k), gen, res)
        if op == "norm":
            s.update(x=_activations((rows, k), gen, DTYPES[case["x"]]),
                     out=torch.empty_like(s["s"]), q=_zeros((rows, k)),
                     sfa=_scales((), rows, k), rstd=_zeros(rows, torch.float32))
        else:
            s.update(rstd=1.0 / torch.sqrt(s["s"].float().square().mean(-1) + EPS),
                     dy=_gradients((rows, k), gen, DTYPES[case["dy"]]),
                     dres=_gradients((rows, k), gen, res), dx=torch.empty_like(s["s"]),
                     dw=_zeros(k, torch.float32))
        return s
    if op in ("dispatch", "combine", "combine_backward"):
        t, g, k, masked = case["tokens"], case["g"], case["k"], case["layout"] == "masked"
        m = case["m"] if masked else capacity(t, case["topk"], g)
        s["ids"], s["weights"] = _router(case, gen)
        s.update(masked=masked, g=g, m=m, lead=(g, m) if masked else (m,))
        ld = (g, m, k) if masked else (m, k)
        lead = (g,) if masked else ()
        if op == "dispatch":
            x = _activations((t, k), gen, torch.bfloat16)
            s["x"], s["sfx"] = _kept(x) if case["x"] == "e4m3" else (x, None)
            s["a"] = _zeros(ld, s["x"].dtype)
            s["sfa"] = None if s["sfx"] is None else _scales(lead, m, k)
            s["group_data"] = _zeros(g if masked else m, torch.int32)
            s["positions"] = _zeros(s["ids"].shape, torch.int32)
            s["counts"] = _zeros(g, torch.int32)
            return s
        s["positions"] = _layout(s["ids"], g, m, masked)[0]
        s["d"] = _activations(ld, gen, torch.bfloat16)
        if op == "combine":
            s["y"] = _zeros((t, k), DTYPES[case["y"]])
        else:
            s.update(dy=_gradients((t, k), gen, DTYPES[case["dy"]]),
                     dd=_zeros(ld, torch.bfloat16) if case["wide"] else None, q=_zeros(ld),
                     sfa=_scales(lead, m, k), dw=_zeros(s["weights"].shape, torch.float32))
        return s
    m, g, layout = case["m"], case["g"], case["layout"]
    s["act"] = case.get("act")
    _rows(s, layout, m, g, seed)
    if op == "columns":
        n = case["n"]
        x = _activations((m, n), gen, torch.float32 if case["x"] == "f32" else torch.bfloat16)
        s["x"], s["sfx"] = _kept(x) if case["x"] == "e4m3" else (x, None)
        padded = (m + 127) // 128 * 128
        s.update(q=_zeros((padded, n)), sf=_zeros((padded // 128, _ld(n)), torch.float32))
        return s
    f = case["f"]
    lead = (g,) if layout == "masked" else ()
    x = _activations((*lead, m, 2 * f), gen, torch.bfloat16)
    if op == "gated":
        s.update(x=x, hq=_zeros((*lead, m, f)), sfh=_scales(lead, m, f))
        s.update(gq=_zeros((*lead, m, 2 * f)) if case["keep"] else None,
                 sfg=_scales(lead, m, 2 * f) if case["keep"] else None)
        return s
    padded = (m + 127) // 128 * 128
    s["x"], s["sfx"] = _kept(x) if case["x"] == "e4m3" else (x, None)
    s.update(dh=_gradients((m, f), gen, torch.bfloat16),
             dq=_zeros((m, 2 * f)), sfd=_scales((), m, 2 * f),
             dqt=_zeros((padded, 2 * f)), sfdt=_zeros((padded // 128, 2 * f), torch.float32),
             hqt=_zeros((padded, f)), sfht=_zeros((padded // 128, f), torch.float32))
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _fp8(q):
    return None if q is None else q.view(torch.float8_e4m3fn)


def _run_own(s):
    import moe_grouped_gemm_block_amd as fp8bs
    op = s["op"]
    if op == "norm":
        fp8bs.fp8bs_rms_norm(s["x"], s["weight"], residual=s["s"], residual_out=s["out"],
                             q=s["q"], sfa=s["sfa"], rstd=s["rstd"], eps=EPS)
        return dict(s=s["out"], q=_fp8(s["q"]), sfa=s["sfa"], rstd=s["rstd"])
    if op == "norm_backward":
        fp8bs.fp8bs_rms_norm_backward(s["s"], s["rstd"], s["weight"], s["dy"], s["dx"],
                                      dresidual=s["dres"], dweight=s["dw"])
        return dict(dx=s["dx"], dw=s["dw"])
    if op == "dispatch":
        fp8bs.fp8bs_moe_dispatch(s["ids"], s["x"], s["a"], s["group_data"], s["positions"],
                                 s["counts"], sfx=s["sfx"], sfa=s["sfa"])
        a = s["a"] if s["sfx"] is None else _fp8(s["a"])
        return dict(a=a, sfa=s["sfa"], group_data=s["group_data"], positions=s["positions"],
                    counts=s["counts"])
    if op == "combine":
        fp8bs.fp8bs_moe_combine(s["d"], s["positions"], s["y"], weights=s["weights"])
        return dict(y=s["y"])
    if op == "combine_backward":
        fp8bs.fp8bs_moe_combine_backward(s["dy"], s["positions"], d=s["d"], weights=s["weights"],
                                         dd=s["dd"], q=s["q"], sfa=s["sfa"], dweights=s["dw"])
        return dict(dd=s["dd"], q=_fp8(s["q"]), sfa=s["sfa"], dw=s["dw"])
    if op == "gated":
        fp8bs.fp8bs_gated_quantize(s["x"], s["hq"], s["sfh"], gq=s["gq"], sfg=s["sfg"],
                                   grouped_layout=s.get("grouped_layout"),
                                   masked_m=s.get("masked_m"), activation=s["act"])
        return dict(hq=_fp8(s["hq"]), sfh=s["sfh"], gq=_fp8(s["gq"]), sfg=s["sfg"])
    if op == "gated_backward":
        fp8bs.fp8bs_gated_quantize_backward(s["x"], s["dh"], sfg=s["sfx"], dq=s["dq"],
                                            sfd=s["sfd"], dqt=s["dqt"], sfdt=s["sfdt"],
                                            hqt=s["hqt"], sfht=s["sfht"],
                                            grouped_layout=s.get("grouped_layout"),
                                            activation=s["act"])
        return dict(dq=_fp8(s["dq"]), sfd=s["sfd"], dqt=_fp8(s["dqt"]), sfdt=s["sfdt"],
                    hqt=_fp8(s["hqt"]), sfht=s["sfht"])
    fp8bs.fp8bs_quantize_128x1(s["x"], s["q"], s["sf"], sfx=s["sfx"],
                               grouped_layout=s.get("grouped_layout"))
    return dict(q=_fp8(s["q"]), sf=s["sf"])


def _quantise(blocks, dim):
    """(e4m3 codes, scales) of f32 values whose blocks lie along `dim`."""
    a = torch.clamp(blocks.abs().amax(dim, keepdim=True), min=1e-4)
    code = torch.clamp(blocks * (448.0 / a), -448.0, 448.0).to(torch.float8_e4m3fn)
    return code, (a / 448.0).squeeze(dim)


def _rows_128(x):
    """1x128: codes [..., rows, k], scales [..., rows, k/128]."""
    code, scale = _quantise(x.view(*x.shape[:-1], x.shape[-1] // 128, 128), -1)
    return code.view(x.shape), scale


def _columns_128(x):
    """128x1: codes [padded][n], scales [padded/128][n]."""
    x = torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % 128))
    code, scale = _quantise(x.view(-1, 128, x.shape[-1]), 1)
    return code.view(x.shape), scale


def _major(scale, valid=None):
    """Scales [..., rows, groups] as they lie; zeros at rows that are not valid."""
    if valid is not None:
        scale = torch.where(valid.unsqueeze(-1), scale, 0.0)
    scale = scale.transpose(-1, -2)
    return torch.nn.functional.pad(scale, (0, -scale.shape[-1] % 4)).contiguous()


def _of_valid(code, valid):
    return torch.where(valid.unsqueeze(-1), code.view(torch.uint8), 0).view(torch.float8_e4m3fn)


def _values(x, sf):
    """float32 values of codes [..., rows, k] and 1x128 scales."""
    v = x.view(torch.float8_e4m3fn).float()
    scale = sf[..., :x.shape[-2]].transpose(-1, -2)
    return (v.view(*x.shape[:-1], -1, 128) * scale.unsqueeze(-1)).view(x.shape)


def _layout(ids, g, m, masked):
    """positions, group data and counts of a router's choices."""
    flat = ids.reshape(-1).long()
    expert = torch.where((flat >= 0) & (flat < g), flat, g)
    order = torch.sort(expert, stable=True).indices
    counts = torch.zeros(g + 1, dtype=torch.int64, device=ids.device)
    counts.scatter_add_(0, expert, torch.ones_like(expert))
    start = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(expert)
    rank[order] = torch.arange(expert.numel(), device=ids.device)
    rank -= start[expert]
    counts = counts[:g]
    if masked:
        row = torch.where((expert < g) & (rank < m), expert * m + rank, -1)
        data = torch.clamp(counts, max=m)
    else:
        padded = (counts + 127) // 128 * 128
        ends = torch.cumsum(padded, 0)
        start = ends - padded
        row = torch.where(expert < g, start[torch.clamp(expert, max=g - 1)] + rank, -1)
        at = torch.arange(m, device=ids.device)
        of = torch.searchsorted(ends, at, right=True)
        inside = torch.clamp(of, max=g - 1)
        data = torch.where((of < g) & (at - start[inside] < counts[inside]), of, -1)
    return row.view(ids.shape).to(torch.int32), data.to(torch.int32), counts.to(torch.int32)


def _scatter(rows, values, positions):
    """[rows, ...]: values of the assignments at their rows, zeros elsewhere."""
    out = torch.zeros((rows + 1, *values.shape[1:]), dtype=values.dtype, device=values.device)
    at = positions.reshape(-1).long()
    out[torch.where(at < 0, rows, at)] = values
    return out[:rows]


def _act(v, name):
    """the activation and its derivative"""
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-v))
        return v * sig, sig * (1.0 + v * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (
        1.0 + 3 * 0.044715 * v * v)


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        v = s["x"].float() + s["s"].float()
        rstd = 1.0 / torch.sqrt(torch.mean(v * v, -1) + EPS)
        code, scale = _rows_128(v * rstd.unsqueeze(-1) * s["weight"].float())
        return dict(s=v.to(s["s"].dtype), q=code, sfa=_major(scale), rstd=rstd)
    if op == "norm_backward":
        xh = s["s"].float() * s["rstd"].unsqueeze(-1)
        dy = s["dy"].float()
        wdy = dy * s["weight"].float()
        mean = torch.mean(wdy * xh, -1, keepdim=True)
        dx = s["dres"].float() + s["rstd"].unsqueeze(-1) * (wdy - xh * mean)
        return dict(dx=dx.to(s["dx"].dtype), dw=torch.sum(dy * xh, 0))
    if op == "dispatch":
        positions, data, counts = _layout(s["ids"], s["g"], s["m"], s["masked"])
        rows = s["g"] * s["m"] if s["masked"] else s["m"]
        token = torch.arange(s["ids"].numel(), device="cuda") // s["ids"].shape[1]
        a = _scatter(rows, s["x"][token], positions).view(*s["lead"], -1)
        sfa = None
        if s["sfx"] is not None:
            scale = s["sfx"].t()[token]
            sfa = _major(_scatter(rows, scale, positions).view(*s["lead"], -1))
            a = a.view(torch.float8_e4m3fn)
        return dict(a=a, sfa=sfa, group_data=data, positions=positions, counts=counts)
    if op in ("combine", "combine_backward"):
        flat = s["d"].view(-1, s["d"].shape[-1])
        here = s["positions"] >= 0
        at = torch.clamp(s["positions"], min=0).long()
    if op == "combine":
        rows = torch.where(here.unsqueeze(-1), flat[at].float(), 0.0)
        return dict(y=torch.sum(rows * s["weights"].unsqueeze(-1), 1).to(s["y"].dtype))
    if op == "combine_backward":
        dy = s["dy"].float().unsqueeze(1)
        dw = torch.where(here, torch.sum(flat[at].float() * dy, -1), 0.0)
        dd = (s["weights"].unsqueeze(-1) * dy).view(-1, flat.shape[-1])
        code, scale = _rows_128(dd)
        code = _scatter(flat.shape[0], code.view(torch.uint8), s["positions"])
        scale = _scatter(flat.shape[0], scale, s["positions"])
        wide = None
        if s["dd"] is not None:
            wide = _scatter(flat.shape[0], dd.to(torch.bfloat16), s["positions"])
            wide = wide.view(s["d"].shape)
        return dict(dd=wide, q=code.view(s["d"].shape).view(torch.float8_e4m3fn),
                    sfa=_major(scale.view(*s["lead"], -1)), dw=dw)
    sfx = s.get("sfx")
    x = s["x"].float() if sfx is None else _values(s["x"], sfx)
    valid = s["valid"]
    if op == "columns":
        code, scale = _columns_128(torch.where(valid.unsqueeze(-1), x, 0.0))
        return dict(q=code, sf=torch.nn.functional.pad(scale, (0, -scale.shape[-1] % 4)))
    gate, up = x.chunk(2, -1)
    act, slope = _act(gate, s["act"])
    if op == "gated":
        code, scale = _rows_128(act * up)
        kept, kept_scale = None, None
        if s["gq"] is not None:
            kept, kept_scale = _rows_128(x)
            kept, kept_scale = _of_valid(kept, valid), _major(kept_scale, valid)
        return dict(hq=_of_valid(code, valid), sfh=_major(scale, valid), gq=kept, sfg=kept_scale)
    dh = s["dh"].float()
    d = torch.where(valid.unsqueeze(-1), torch.cat((dh * up * slope, dh * act), -1), 0.0)
    h = torch.where(valid.unsqueeze(-1), act * up, 0.0)
    (dq, sfd), (dqt, sfdt), (hqt, sfht) = _rows_128(d), _columns_128(d), _columns_128(h)
    return dict(dq=dq, sfd=_major(sfd, valid), dqt=dqt, sfdt=sfdt, hqt=hqt, sfht=sfht)


# ---- the definition in 64 bits ------------------------------------------------

def _e4m3(v):
    """nearest e4m3 value of magnitudes up to 448"""
    top = torch.where(v == 0, 1.0, v.abs())
    e = torch.floor(torch.log2(top))
    e = torch.where(2.0 ** e > top, e - 1, torch.where(2.0 ** (e + 1) <= top, e + 1, e))
    step = 2.0 ** (torch.clamp(e, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_blocks(x, dim):
    """codes' values and scales of x, blocks of 128 along dim (0 or -1 of a matrix)"""
    if dim == 0:
        code, scale = _exact_blocks(x.t(), -1)
        return code.t(), scale.t()
    b = x.reshape(x.shape[0], -1, 128)
    top = b.abs().max(-1).values.clamp(min=1e-4)
    return _e4m3(b / top[..., None] * 448).reshape(x.shape), top / 448


def _exact_scales(scale, slots):
    """scales [slots * rows, groups] as they lie, per slot"""
    rows = scale.shape[0] // slots
    out = torch.zeros(slots, scale.shape[1], _ld(rows), dtype=torch.float64, device="cuda")
    out[..., :rows] = scale.view(slots, rows, -1).permute(0, 2, 1)
    return out


def _exact_kept(x, sf):
    if sf is None:
        return x.double()
    n = x.to(torch.int32)
    mant, expo = (n % 8).double(), ((n // 8) % 16).double()
    v = torch.where(expo == 0, mant * 2.0 ** -9, (1 + mant / 8) * 2.0 ** (expo - 7))
    v = torch.where(n >= 128, -v, v)
    return v * torch.repeat_interleave(sf.double().t()[:x.shape[0]], 128, 1)


def _exact_act(v, name):
    if name == "silu":
        sig = torch.sigmoid(v)
        return v * sig, sig + v * sig * (1 - sig)
    inner = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    t = torch.tanh(inner)
    return 0.5 * v * (1 + t), (0.5 + 0.5 * t + 0.5 * v * (1 - t ** 2) * math.sqrt(2 / math.pi)
                               * (1 + 0.134145 * v ** 2))


def _exact_layout(s):
    """positions [tokens][topk], each expert's count, and the rows' experts"""
    ids, g, m = s["ids"].tolist(), s["g"], s["m"]
    counts = [0] * g
    ranks = []
    for row in ids:
        ranks.append([])
        for e in row:
            ranks[-1].append(counts[e] if 0 <= e < g else -1)
            if 0 <= e < g:
                counts[e] += 1
    start, owner = [], []
    for e in range(g):
        if s["masked"]:
            start.append(e * m)
        else:
            start.append(len(owner))
            owner += [e] * counts[e] + [-1] * (-counts[e] % 128)
    owner += [-1] * (0 if s["masked"] else m - len(owner))
    positions = [[-1 if r < 0 or (s["masked"] and r >= m) else start[e] + r
                  for e, r in zip(row, rank)] for row, rank in zip(ids, ranks)]
    data = [min(c, m) for c in counts] if s["masked"] else owner
    return (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (positions, data, counts))


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        v = s["x"].double() + s["s"].double()
        rstd = (v.pow(2).sum(-1) / v.shape[-1] + EPS).rsqrt()
        code, scale = _exact_blocks(v * rstd[:, None] * s["weight"].double(), -1)
        return dict(s=v, q=code, sfa=_exact_scales(scale, 1)[0], rstd=rstd)
    if op == "norm_backward":
        r, w, dy = s["rstd"].double()[:, None], s["weight"].double(), s["dy"].double()
        v = s["s"].double()
        dot = (v * w * dy).sum(-1, keepdim=True) / v.shape[-1]
        return dict(dx=s["dres"].double() + w * dy * r - v * r ** 3 * dot,
                    dw=(dy * v * r).sum(0))
    if op == "dispatch":
        positions, data, counts = _exact_layout(s)
        slots = s["g"] if s["masked"] else 1
        a = torch.zeros(slots * s["m"], case["k"], dtype=torch.float64, device="cuda")
        scale = torch.zeros(slots * s["m"], case["k"] // 128, dtype=torch.float64, device="cuda")
        x = s["x"] if s["sfx"] is None else s["x"].view(torch.float8_e4m3fn)
        for j in range(positions.shape[1]):
            t = torch.nonzero(positions[:, j] >= 0)[:, 0]
            a[positions[t, j].long()] = x[t].double()
            if s["sfx"] is not None:
                scale[positions[t, j].long()] = s["sfx"].double()[:, t].t()
        sfa = None if s["sfx"] is None else _exact_scales(scale, slots).reshape(s["sfa"].shape)
        return dict(a=a.reshape(s["a"].shape), sfa=sfa, group_data=data, positions=positions,
                    counts=counts)
    if op in ("combine", "combine_backward"):
        flat = s["d"].reshape(-1, case["k"])
        positions, w = s["positions"], s["weights"].double()
        out = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w)
        dd = torch.zeros(flat.shape, dtype=torch.float64, device="cuda")
        code = torch.zeros_like(dd)
        scale = torch.zeros(flat.shape[0], case["k"] // 128, dtype=torch.float64, device="cuda")
        for j in range(positions.shape[1]):
            t = torch.nonzero(positions[:, j] >= 0)[:, 0]
            if t.numel() == 0:
                continue
            row = positions[t, j].long()
            if op == "combine":
                out[t] += w[t, j, None] * flat[row].double()
                continue
            dy = s["dy"][t].double()
            dw[t, j] = (dy * flat[row].double()).sum(-1)
            dd[row] = w[t, j, None] * dy
            code[row], scale[row] = _exact_blocks(dd[row], -1)
        if op == "combine":
            return dict(y=out)
        shape = s["d"].shape
        sfa = _exact_scales(scale, s["g"] if s["masked"] else 1).reshape(s["sfa"].shape)
        return dict(dd=dd.reshape(shape) if case["wide"] else None, q=code.reshape(shape),
                    sfa=sfa, dw=dw)
    valid = s["valid"].reshape(-1, 1)
    slots = case["g"] if case["layout"] == "masked" else 1
    x = s["x"].reshape(-1, s["x"].shape[-1])
    x = _exact_kept(x, s.get("sfx"))
    live = valid.double()

    def columns(v):
        more = torch.zeros(-v.shape[0] % 128, v.shape[1], dtype=v.dtype, device="cuda")
        return _exact_blocks(torch.cat((torch.where(valid, v, 0.0), more)), 0)

    if op == "columns":
        code, scale = columns(x)
        return dict(q=code, sf=scale)
    f = case["f"]
    value, slope = _exact_act(x[:, :f], s["act"])
    up = x[:, f:]
    if op == "gated":
        code, scale = _exact_blocks(value * up, -1)
        got = dict(hq=(code * live).reshape(s["hq"].shape),
                   sfh=_exact_scales(scale * live, slots).reshape(s["sfh"].shape), gq=None,
                   sfg=None)
        if case["keep"]:
            code, scale = _exact_blocks(x, -1)
            got.update(gq=(code * live).reshape(s["gq"].shape),
                       sfg=_exact_scales(scale * live, slots).reshape(s["sfg"].shape))
        return got
    dh = s["dh"].double()
    d = torch.cat((dh * up * slope, dh * value), 1)
    code, scale = _exact_blocks(d, -1)
    dqt, sfdt = columns(d)
    hqt, sfht = columns(value * up)
    return dict(dq=code * live, sfd=_exact_scales(scale * live, 1)[0], dqt=dqt, sfdt=sfdt,
                hqt=hqt, sfht=sfht)
