"""What is measured of the MXFP4 operators: the quantiser with its inverse, the block-scaled
product, the gated feed-forward block, its backward pass, and a whole feed-forward layer.

MXFP4 here: 32 consecutive values along K share one power-of-two scale 2^(e - 127) with an
8-bit exponent e (E8M0), e - 127 = floor(log2(largest magnitude)) - 2; each value is held as
a 4-bit e2m1 number (0, .5, 1, 1.5, 2, 3, 4, 6 with a sign; nearest, ties to the even code,
magnitudes above 6 saturate).  Codes lie two to a byte, the even K position in the low
nibble: uint8 [rows][k/2].  Exponents lie four to an int32, K-group-major:
int32 [k/128][ld], ld = rows rounded up to a multiple of 4; byte j of word (c, r) is the
exponent of row r's values 128c + 32j .. 128c + 32j + 31.

The weight of a gated block holds the gate rows 0 .. f-1 and the up rows f .. 2f-1;
h = act(x Wg^T) * (x Wu^T).

Grouped inputs: "contiguous" concatenates the experts' rows, each expert's segment padded to
a multiple of 128 rows, with an expert index per row (-1: padding); "masked" gives every
expert a slot of max_m rows of which the first masked_m are valid.  Rows that are not valid
are not written; the outputs' buffers start as zeros.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # activations of a decode step of 64 sequences, quantised and read back
        dict(name="round trip 64x7168", op="round_trip", rows=64, k=7168, dtype="bf16"),
        # a prefill batch routed to eight experts, before its expert products
        dict(name="round trip 33152x7168", op="round_trip", rows=33152, k=7168, dtype="bf16"),
        # one token against one projection: the smallest call, latency counts
        dict(name="product 1x4096x7168", op="product", layout="dense", m=1, n=4096, k=7168, g=1),
        # a decode batch, N no multiple of 128
        dict(name="product 128x2112x7168", op="product", layout="dense", m=128, n=2112, k=7168,
             g=1),
        # a prefill chunk against a long-K projection
        dict(name="product 4096x7168x16384", op="product", layout="dense", m=4096, n=7168,
             k=16384, g=1),
        # expert down projections of a decode step, ragged slots
        dict(name="product masked g16", op="product", layout="masked", m=256, n=7168, k=2048,
             g=16),
        # odd sizes, the other activation
        dict(name="gated 333x1056x1536", op="gated", layout="dense", m=333, f=1056, k=1536, g=1,
             act="gelu_tanh"),
        # gate and up projections of a prefill batch over eight experts
        dict(name="gated contiguous g8", op="gated", layout="contiguous", m=33280, f=2048,
             k=7168, g=8, act="silu"),
        # a whole feed-forward layer on a decode batch: quantise, gated block with its output
        # quantised, down projection
        dict(name="layer 64x2048x7168", op="layer", layout="dense", m=64, f=2048, k=7168, g=1,
             act="silu"),
        # the same over sixteen experts' slots
        dict(name="layer masked g16", op="layer", layout="masked", m=256, f=2048, k=7168, g=16,
             act="silu"),
        # the gradients of a small ragged block
        dict(name="backward 200x416x640", op="backward", layout="dense", m=200, f=416, k=640,
             g=1, act="gelu_tanh"),
        # a training step's gradients over eight experts
        dict(name="backward contiguous g8", op="backward", layout="contiguous", m=16384, f=2048,
             k=7168, g=8, act="silu"),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        """log-uniform over lo .. hi, a multiple of step"""
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        v = max(step, int(round(v / step)) * step)
        return v - step if v == 3072 else v

    op = rng.choice(["round_trip", "product", "product", "gated", "gated", "layer", "backward",
                     "backward"])
    if op == "round_trip":
        return dict(op=op, rows=size(1, 30000), k=size(128, 7168, 128),
                    dtype=rng.choice(["bf16", "f32"]))
    layout = rng.choice(["dense", "contiguous"] + ([] if op == "backward" else ["masked"]))
    c = dict(op=op, layout=layout)
    if layout == "dense":
        c.update(m=size(1, 4096), g=1)
    elif layout == "contiguous":
        c.update(m=size(128, 16384, 128), g=size(1, 16))
    else:
        c.update(m=size(1, 400), g=size(1, 16))
    if op == "product":
        c.update(n=size(16, 7168), k=size(128, 7168, 128))
    else:
        step = 128 if op == "layer" else 32
        c.update(f=size(step, 2048, step), k=size(128, 7168, 128),
                 act=rng.choice(["silu", "gelu_tanh"]))
    return c


def work(case):
    op = case["op"]
    packed = 0.5 + 1.0 / 32.0                       # bytes of one MXFP4 value
    if op == "round_trip":
        n = case["rows"] * case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (size + 2 * packed + 2), "flops": 2.0 * n}
    g, k = case["g"], case["k"]
    # rows that hold a token, as prepare() fills them on average
    rows = case["m"]
    if case["layout"] == "contiguous":
        rows = max(1, case["m"] - 64 * min(g, case["m"] // 128))
    elif case["layout"] == "masked":
        rows = g * (case["m"] + 1) // 2
    if op == "product":
        n = case["n"]
        return {"bytes": packed * k * (rows + g * n) + 2.0 * rows * n,
                "flops": 2.0 * rows * n * k}
    f = case["f"]
    if op == "gated":
        return {"bytes": packed * k * (rows + 2 * g * f) + 2.0 * rows * f,
                "flops": 4.0 * rows * f * k}
    if op == "layer":
        return {"bytes": 2.0 * rows * k + packed * 3 * g * f * k + 2.0 * rows * k,
                "flops": 6.0 * rows * f * k}
    return {"bytes": packed * k * (rows + 2 * g * f) + 2.0 * rows * (f + k) + 4.0 * g * f * k,
            "flops": 12.0 * rows * f * k}


# ---- inputs ----------------------------------------------------------------

def _pack(x):
    """Codes and exponents of x [..., rows, k] in the layout described above."""
    rows, k = x.shape[-2], x.shape[-1]
    code, e = _codes(x.float())
    code = code.to(torch.uint8).view(*x.shape[:-1], k // 2, 2)
    q = code[..., 0] | (code[..., 1] << 4)
    ld = (rows + 3) // 4 * 4
    sf = torch.zeros(*x.shape[:-2], k // 128, ld, 4, dtype=torch.uint8, device=x.device)
    sf[..., :rows, :] = e.to(torch.uint8).view(*x.shape[:-1], k // 128, 4).transpose(-2, -3)
    return q.contiguous(), sf.view(torch.int32).squeeze(-1).contiguous()


def _codes(x):
    """4-bit codes and biased exponents of float32 values."""
    blocks = x.view(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = blocks.abs().amax(-1)
    e = torch.clamp(torch.frexp(amax).exponent - 3, -127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    v = blocks * _power(127 - e).unsqueeze(-1)
    a = v.abs()
    code = ((a > 0.25).to(torch.int8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    return (code + 8 * torch.signbit(v).to(torch.int8)).view(x.shape), e + 127


def _power(e):
    """2^(e - 127) in float32, from its bits (e = 0: the subnormal 2^-127)"""
    return torch.where(e > 0, e << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _activations(shape, gen, dtype=torch.bfloat16):
    """Hidden states: unit variance, tokens of different size, a few large channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    size = torch.exp(0.3 * torch.randn(shape[:-1], generator=gen, device="cuda"))
    channel = torch.where(torch.rand(shape[-1], generator=gen, device="cuda") < 0.01, 6.0, 1.0)
    return (x * size.unsqueeze(-1) * channel).to(dtype)


def _weights(shape, gen):
    return _pack(torch.randn(shape, generator=gen, device="cuda") / math.sqrt(shape[-1]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "round_trip":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        return dict(op=op, x=_activations((case["rows"], case["k"]), gen, dtype))
    layout, m, g, k = case["layout"], case["m"], case["g"], case["k"]
    s = dict(op=op, layout=layout, act=case.get("act"))
    host = torch.Generator().manual_seed(seed)
    if layout == "masked":
        s["masked_m"] = torch.randint(0, m + 1, (g,), generator=host).to(torch.int32).cuda()
        s["expected_m"] = (m + 1) // 2
        s["valid"] = torch.arange(m, device="cuda")[None, :] < s["masked_m"][:, None]
    elif layout == "contiguous":
        # cut the 128-row blocks at random places into one run per expert (empty ones too);
        # the last block of a run ends in up to 127 rows of padding
        blocks = m // 128
        cuts = torch.randint(0, blocks + 1, (g - 1,), generator=host).sort().values.tolist()
        at = [128 * b for b in [0] + cuts + [blocks]]
        pad = torch.randint(0, 128, (g,), generator=host).tolist()
        s["segments"] = [(a, b - p if b > a else b) for a, b, p in zip(at[:-1], at[1:], pad)]
        index = torch.full((m,), -1, dtype=torch.int32)
        for e, (a, b) in enumerate(s["segments"]):
            index[a:b] = e
        s["grouped_layout"] = index.cuda()
        s["valid"] = s["grouped_layout"] >= 0
    else:
        s["segments"] = [(0, m)]
    xs = (g, m, k) if layout == "masked" else (m, k)
    lead = () if layout == "dense" else (g,)
    if op == "layer":
        s["x"] = _activations(xs, gen)
    else:
        s["a"], s["sfa"] = _pack(_activations(xs, gen))
    cols = case["n"] if op == "product" else 2 * case["f"]
    s["b"], s["sfb"] = _weights(lead + (cols, k), gen)
    if op == "layer":
        s["b2"], s["sfb2"] = _weights(lead + (k, case["f"]), gen)
    if op == "backward":
        f = case["f"]
        s["dh"] = (torch.randn(xs[:-1] + (f,), generator=gen, device="cuda")
                   * 0.05).to(torch.bfloat16)
        s["da"] = torch.zeros(xs, dtype=torch.bfloat16, device="cuda")
        s["db"] = torch.zeros(lead + (cols, k), dtype=torch.bfloat16, device="cuda")
    else:
        width = {"product": case.get("n"), "gated": case.get("f"), "layer": k}[op]
        s["d"] = torch.zeros(xs[:-1] + (width,), dtype=torch.bfloat16, device="cuda")
    return s


# ---- one pass --------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import moe_grouped_gemm_block_amd as fp8bs
    op = s["op"]
    if op == "round_trip":
        q, sf = fp8bs.quantize_mxfp4(s["x"])
        return fp8bs.dequantize_mxfp4(q, sf)
    layout = s["layout"]
    if op == "product":
        ops = (s["a"], s["sfa"], s["b"], s["sfb"], s["d"])
        if layout == "dense":
            fp8bs.fp8bs_dense_nt_mxfp4(*ops)
        elif layout == "contiguous":
            fp8bs.fp8bs_grouped_contiguous_nt_mxfp4(*ops, s["grouped_layout"])
        else:
            fp8bs.fp8bs_grouped_masked_nt_mxfp4(*ops, s["masked_m"], expected_m=s["expected_m"])
        return s["d"]
    if op == "gated":
        ops = (s["a"], s["sfa"], s["b"], s["sfb"], s["d"])
        if layout == "dense":
            fp8bs.fp8bs_gated_dense_mxfp4(*ops, activation=s["act"])
        elif layout == "contiguous":
            fp8bs.fp8bs_gated_contiguous_mxfp4(*ops, s["grouped_layout"], activation=s["act"])
        else:
            fp8bs.fp8bs_gated_masked_mxfp4(*ops, s["masked_m"], expected_m=s["expected_m"],
                                           activation=s["act"])
        return s["d"]
    if op == "layer":
        w = (s["b"], s["sfb"], s["b2"], s["sfb2"])
        if layout == "dense":
            fp8bs.feed_forward_mxfp4(s["x"], *w, activation=s["act"], out=s["d"])
        elif layout == "contiguous":
            fp8bs.feed_forward_mxfp4(s["x"], *w, activation=s["act"], out=s["d"],
                                     grouped_layout=s["grouped_layout"])
        else:
            fp8bs.feed_forward_mxfp4(s["x"], *w, activation=s["act"], out=s["d"],
                                     masked_m=s["masked_m"], expected_m=s["expected_m"])
        return s["d"]
    ops = (s["a"], s["sfa"], s["b"], s["sfb"], s["dh"], s["da"], s["db"])
    if layout == "dense":
        fp8bs.fp8bs_gated_dense_mxfp4_backward(*ops, activation=s["act"])
    else:
        fp8bs.fp8bs_gated_contiguous_mxfp4_backward(*ops, s["grouped_layout"],
                                                    activation=s["act"])
    return {"da": s["da"], "db": s["db"]}


def _decode(q, sf):
    """float32 values of packed codes and exponents."""
    rows = q.shape[-2]
    codes = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    e = sf.unsqueeze(-1).view(torch.uint8)[..., :rows, :].transpose(-2, -3).flatten(-2)
    v = table[codes.int()].view(*codes.shape[:-1], -1, 32)
    return (v * _power(e.int()).unsqueeze(-1)).view(codes.shape)


def _round_trip(x):
    """float32 values that x's MXFP4 form stands for."""
    code, e = _codes(x.float())
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=x.device)
    v = table[code.int()].view(*x.shape[:-1], -1, 32)
    return (v * _power(e).unsqueeze(-1)).view(x.shape)


def _act(v, name):
    """the activation and its derivative"""
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-v))
        return v * sig, sig * (1.0 + v * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (
        1.0 + 3 * 0.044715 * v * v)


def _times(s, x, w):
    """x W^T, each row with its expert's W [g][n][k]; zeros at rows that are not valid."""
    if s["layout"] == "masked":
        y = torch.matmul(x, w.transpose(-1, -2).contiguous())
        return torch.where(s["valid"].unsqueeze(-1), y, 0.0)
    if s["layout"] == "dense":
        return x @ w.t()
    y = x.new_zeros(x.shape[0], w.shape[1])
    [torch.matmul(x[a:b], w[e].t(), out=y[a:b]) for e, (a, b) in enumerate(s["segments"])]
    return y


def _gate(s, x, w):
    gate, up = _times(s, x, w).chunk(2, -1)
    return _act(gate, s["act"])[0] * up


def _run_plain(s):
    op = s["op"]
    if op == "round_trip":
        return _round_trip(s["x"]).to(torch.bfloat16)
    if op == "layer":
        x = _round_trip(s["x"])
    else:
        x = _decode(s["a"], s["sfa"])
    w = _decode(s["b"], s["sfb"])
    if op == "product":
        return _times(s, x, w).to(torch.bfloat16)
    if op == "gated":
        return _gate(s, x, w).to(torch.bfloat16)
    if op == "layer":
        h = _round_trip(_gate(s, x, w))
        return _times(s, h, _decode(s["b2"], s["sfb2"])).to(torch.bfloat16)
    gate, up = _times(s, x, w).chunk(2, -1)
    act, slope = _act(gate, s["act"])
    dh = s["dh"].float()
    d = torch.cat((dh * up * slope, dh * act), -1)
    w = w if w.dim() == 3 else w[None]
    da = torch.zeros_like(x)
    [torch.matmul(d[a:b], w[e], out=da[a:b]) for e, (a, b) in enumerate(s["segments"])]
    db = torch.stack([d[a:b].t() @ x[a:b] for a, b in s["segments"]]).view(s["db"].shape)
    return {"da": da.to(torch.bfloat16), "db": db.to(torch.bfloat16)}


# ---- the definition in 64 bits ------------------------------------------------

def _exact_values(q, sf):
    low, high = (q % 16).double(), (q // 16).double()
    n = torch.stack((low, high), -1).reshape(*q.shape[:-1], 2 * q.shape[-1])
    sign = 1.0 - 2.0 * (n >= 8)
    n = n % 8
    v = torch.where(n < 2, n / 2, (1 + (n % 2) / 2) * 2.0 ** (torch.floor(n / 2) - 1))
    rows, words = q.shape[-2], sf.shape[-2]
    e = torch.stack([torch.bitwise_and(sf >> (8 * j), 255) for j in range(4)], -1)[..., :rows, :]
    e = torch.movedim(e, -2, -3).reshape(*q.shape[:-1], 4 * words).double()
    return sign * v * torch.repeat_interleave(2.0 ** (e - 127), 32, -1)


def _exact_rounded(x):
    x = x.double()
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(2.0 ** e > top, e - 1, e)
    e = torch.where(2.0 ** (e + 1) <= top, e + 1, e)
    scale = 2.0 ** torch.clamp(e - 2, min=-127)
    a = b.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.clamp(torch.round(a / step) * step, max=6.0)
    return (torch.sign(b) * a * scale).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "round_trip":
        return _exact_rounded(s["x"])
    g, m = case["g"], case["m"]
    x = _exact_rounded(s["x"]) if op == "layer" else _exact_values(s["a"], s["sfa"])
    flat = x.reshape(-1, x.shape[-1])
    if s["layout"] == "masked":
        counts = s["masked_m"].tolist()
        runs = [(e * m, e * m + counts[e]) for e in range(g)]
    else:
        runs = s["segments"]

    def experts(q, sf):
        return (q[None], sf[None]) if q.dim() == 2 else (q, sf)

    def slope_and_value(v):
        if s["act"] == "silu":
            sig = torch.sigmoid(v)
            return sig + v * sig * (1 - sig), v * sig
        inner = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        sech2 = 1 / torch.cosh(inner) ** 2
        t = torch.tanh(inner)
        return (0.5 + 0.5 * t + 0.5 * v * sech2 * math.sqrt(2 / math.pi)
                * (1 + 0.134145 * v ** 2)), 0.5 * v * (1 + t)

    b, sfb = experts(s["b"], s["sfb"])
    if op == "backward":
        f = case["f"]
        da = torch.zeros(flat.shape, dtype=torch.float64, device="cuda")
        db = torch.zeros(b.shape[0], 2 * f, case["k"], dtype=torch.float64, device="cuda")
        dh = s["dh"].double()
        for e, (lo, hi) in enumerate(runs):
            w = _exact_values(b[e], sfb[e])
            xe = flat[lo:hi]
            gate, up = xe @ w[:f].t(), xe @ w[f:].t()
            slope, value = slope_and_value(gate)
            dg, du = dh[lo:hi] * up * slope, dh[lo:hi] * value
            da[lo:hi] = dg @ w[:f] + du @ w[f:]
            db[e, :f] = dg.t() @ xe
            db[e, f:] = du.t() @ xe
        return {"da": da, "db": db.reshape(s["db"].shape)}
    out = torch.zeros(flat.shape[0], s["d"].shape[-1], dtype=torch.float64, device="cuda")
    if op == "layer":
        b2, sfb2 = experts(s["b2"], s["sfb2"])
    for e, (lo, hi) in enumerate(runs):
        w = _exact_values(b[e], sfb[e])
        y = flat[lo:hi] @ w.t()
        if op != "product":
            f = case["f"]
            y = slope_and_value(y[:, :f])[1] * y[:, f:]
        if op == "layer" and hi > lo:
            y = _exact_rounded(y) @ _exact_values(b2[e], sfb2[e]).t()
        if hi > lo:
            out[lo:hi] = y
    return out.reshape(s["d"].shape)
