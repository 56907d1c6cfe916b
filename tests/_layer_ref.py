"""Plain references of the operators between the FP8 products (numpy on the CPU): definitions in
64 bits, and the quantisers bit for bit (each step one IEEE operation in 32 bits)."""
import numpy as np
import torch

F32, F64 = np.float32, np.float64
E = 2.0 ** -24                     # bound of an FP32 rounding, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def bf16(x):
    """float32 values rounded to bf16, as float32"""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=F32)).to(torch.bfloat16).float().numpy()


def host(t):
    """a tensor's values: float32 for bf16, codes as uint8"""
    t = t.detach().cpu()
    if t.dtype == torch.bfloat16:
        return t.float().numpy()
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8).numpy()
    return t.numpy()


# ---- e4m3 -----------------------------------------------------------------------

_c = np.arange(256)
_mag = np.where((_c & 127) >> 3 == 0, (_c & 7) * 2.0 ** -9,
                (1 + (_c & 7) / 8) * 2.0 ** (((_c & 127) >> 3) - 7.0))
VALUES = np.where(_c & 128, -_mag, _mag)
VALUES[[127, 255]] = np.nan
_POSITIVE = VALUES[:127]
# midpoints between neighbouring magnitudes
_MID = (_POSITIVE[1:] + _POSITIVE[:-1]) / 2


def codes(v):
    """e4m3 codes of float32 values of magnitude at most 448 or a rounding more: nearest, ties to
    the even code; NaN gives 127"""
    v = np.asarray(v, dtype=F64)
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    up = np.searchsorted(_MID, a, side="left")         # ties: the lower code
    tie = (up < 126) & (a == _MID[np.minimum(up, 125)])
    c = up + (tie & (up % 2 == 1))
    c = np.where(np.isnan(v), 127, c | (np.signbit(v) * 128))
    return c.astype(np.uint8)


def quantise(x, axis):
    """codes and scales of float32 values, blocks of 128 along axis (0 or -1 of a matrix)"""
    x = np.ascontiguousarray(x, dtype=F32)
    if axis == 0:
        c, s = quantise(x.T, -1)
        return np.ascontiguousarray(c.T), np.ascontiguousarray(s.T)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 128, 128)
    a = np.abs(b)
    a = np.where(np.isnan(a), F32(0), a).max(-1)
    a = np.maximum(a, F32(1e-4))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        inv = (F32(448) / a).astype(F32)
        scale = (a / F32(448)).astype(F32)
        q = codes((b * inv[..., None]).astype(F32))
    return q.reshape(x.shape), scale


def same_codes(got, want):
    """equal codes; a NaN's may have either sign"""
    got, want = np.asarray(got), np.asarray(want)
    return np.array_equal(np.where(got & 127 == 127, 127, got), np.where(want & 127 == 127, 127, want))


def row_scales(sf, rows):
    """[.., groups, ld] -> [.., rows, groups]"""
    return np.swapaxes(host(sf), -1, -2)[..., :rows, :]


def values_1x128(q, sf):
    """64-bit values of codes [.., rows, k] and 1x128 scales"""
    q = host(q)
    return VALUES[q] * np.repeat(row_scales(sf, q.shape[-2]).astype(F64), 128, -1)


def values_128x1(q, sf):
    q = host(q)
    return VALUES[q] * np.repeat(host(sf)[:, :q.shape[1]].astype(F64), 128, 0)


def check_quantised(q, scale, want, tol, axis, what):
    """codes and scales [rows, k / 128] (axis 0: [rows / 128, n]) against 64-bit values `want`, of
    which the quantised ones are off by at most tol (an array): the scale is the largest
    magnitude's to two roundings, a value within half a step of e4m3 -- 2^-4 of it, or 2^-10 of the
    scale below 2^-6 -- and the roundings of the factor and the product (3 E)."""
    if axis == 0:
        q, scale, want, tol = q.T, scale.T, want.T, tol.T
    block = lambda x: x.reshape(*x.shape[:-1], x.shape[-1] // 128, 128)  # noqa: E731
    top = np.maximum(np.abs(block(want)).max(-1), 1e-4)
    off = block(tol).max(-1)
    assert np.all(np.abs(scale * 448.0 - top) <= off + 3 * E * top), what
    s = np.repeat(scale.astype(F64), 128, -1)
    got = VALUES[q] * s
    half = np.maximum(np.abs(want) * 2.0 ** -4, s * 2.0 ** -10)
    bad = np.abs(got - want) > half + tol * (1 + 2.0 ** -4) + 4 * E * np.abs(want) + 1e-30
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


# ---- activation -------------------------------------------------------------------

def activation(v, act):
    """(act, act', and how far 32-bit evaluations of both may be off).  The logistic function s
    and 1 - s: exponential and reciprocal within 2 units each (4 E), the argument's roundings as
    relative errors of the exponential, |argument| times as large (its own product is
    compensated).  act = v s then has s's error and one rounding; act' = s + act (1 - s) [...]
    the errors of its terms' magnitudes.  s below 2^-126 is no normal number: its reciprocal
    instruction gives 0 there, off by at most 2^-126, which act multiplies by |v| and act' by
    1 + |v| (gelu: times the derivative of its argument, 210 at v = -10).  Twice that covers the
    roundings of what it is multiplied with."""
    with np.errstate(over="ignore", invalid="ignore"):
        if act == "silu":
            s = 1 / (1 + np.exp(-v))
            rest = 1 / (1 + np.exp(v))
            rel = 12 * E
            value, slope = v * s, s + v * s * rest
            size, reach = s + np.abs(v) * s * rest, 1 + np.abs(v)
        else:
            c = np.sqrt(2 / np.pi)
            y2 = 2 * c * (v + 0.044715 * v ** 3)
            s = 1 / (1 + np.exp(-y2))
            rest = 1 / (1 + np.exp(y2))
            rel = (12 + 8 * np.minimum(np.abs(y2), 110)) * E
            t = 2 * c * (1 + 0.134145 * v * v)
            value, slope = v * s, s + v * s * rest * t
            size, reach = s + np.abs(v) * s * rest * t, 1 + np.abs(v) * t
    tiny = 2.0 ** -125
    return value, slope, np.abs(value) * rel + np.abs(v) * tiny, size * (2 * rel + 8 * E) + reach * tiny


# ---- layouts ----------------------------------------------------------------------

def layout_of(ids, groups, m, masked):
    """positions, group data, counts, and the rows' tokens (-1), by hand"""
    counts = [0] * groups
    rank = np.full(ids.shape, -1, np.int64)
    for t, row in enumerate(ids.tolist()):
        for j, e in enumerate(row):
            if 0 <= e < groups:
                rank[t, j] = counts[e]
                counts[e] += 1
    start, at = [], 0
    for e in range(groups):
        start.append(e * m if masked else at)
        at += (counts[e] + 127) // 128 * 128
    rows = groups * m if masked else m
    positions = np.full(ids.shape, -1, np.int32)
    token = np.full(rows, -1, np.int64)
    data = np.array([min(c, m) for c in counts] if masked else [-1] * m, np.int32)
    for (t, j), r in np.ndenumerate(rank):
        if r < 0 or (masked and r >= m):
            continue
        row = start[int(ids[t, j])] + r
        positions[t, j] = row
        token[row] = t
        if not masked:
            data[row] = ids[t, j]
    return positions, data, np.array(counts, np.int32), token


def contiguous_layout(counts, m=None):
    """grouped_layout of experts with so many rows, and the K-grouped sizes"""
    out = []
    for e, c in enumerate(counts):
        out += [e] * c + [-1] * (-c % 128)
    ks = [(c + 127) // 128 * 128 for c in counts]
    out += [-1] * ((len(out) if m is None else m) - len(out))
    return np.array(out, np.int32), ks
