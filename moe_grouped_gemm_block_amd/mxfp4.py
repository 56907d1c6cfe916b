"""MXFP4 operators: quantiser and its inverse, block-scaled product, gated feed-forward block
and its backward pass, and a feed-forward layer made of them.

Binding of the ``fp8bs_*_mxfp4`` calls of ``libfp8bs.so`` (``include/fp8bs.h`` states the
formats, the formulas and the valid rows); argument checks and marshalling only.

A quantised matrix is a pair: codes, uint8 (or ``torch.float4_e2m1fn_x2``) ``[..., rows,
k/2]``, and exponents, int32 ``[..., k/128, get_sfa_ld(rows)]``.  Outputs are written in
place at valid rows; ``quantize_mxfp4``, ``dequantize_mxfp4`` and ``feed_forward_mxfp4``
allocate what they return.
"""
from __future__ import annotations

import ctypes

import moe_grouped_gemm_block_amd as _pkg
from moe_grouped_gemm_block_amd import (FP8BSError, LAYOUT_CONTIGUOUS, LAYOUT_DENSE, LAYOUT_MASKED,
                                        _dev_ptr, _torch)

__all__ = [
    "fp8bs_quantize_mxfp4", "fp8bs_dequantize_mxfp4", "quantize_mxfp4", "dequantize_mxfp4",
    "fp8bs_dense_nt_mxfp4", "fp8bs_grouped_contiguous_nt_mxfp4", "fp8bs_grouped_masked_nt_mxfp4",
    "fp8bs_gated_dense_mxfp4", "fp8bs_gated_contiguous_mxfp4", "fp8bs_gated_masked_mxfp4",
    "fp8bs_gated_dense_mxfp4_q", "fp8bs_gated_contiguous_mxfp4_q", "fp8bs_gated_masked_mxfp4_q",
    "fp8bs_gated_dense_mxfp4_backward", "fp8bs_gated_contiguous_mxfp4_backward",
    "gated_backward_workspace_size", "fp8bs_feed_forward_mxfp4", "feed_forward_workspace_size",
    "feed_forward_mxfp4", "ACTIVATIONS",
]

ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}

_lib = None


def _load():
    """The library with this module's prototypes, and torch's types and queries (torch is
    imported at the first call, like the library)."""
    global _lib, _Tensor, _empty, _device_index, _raw_stream
    global _FP4, _INT32, _FLOAT, _BF16, _UINT8, _bf16, _f32, _u8, _i32
    if _lib is not None:
        return _lib
    lib = _pkg._load()
    torch = _torch()
    _Tensor, _empty = torch.Tensor, torch.empty
    _device_index = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
        else torch.cuda.current_device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _bf16, _f32, _u8, _i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    packed = getattr(torch, "float4_e2m1fn_x2", None)
    _FP4 = (_u8,) if packed is None else (_u8, packed)
    _INT32, _FLOAT, _UINT8 = (_i32,), (_bf16, _f32), (_u8,)
    _BF16 = _pkg._bf16_dtypes()
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    for name, args in {
        "fp8bs_quantize_mxfp4": [P, I, P, P, I, I, I, P],
        "fp8bs_dequantize_mxfp4": [P, P, P, I, I, I, I, P],
        "fp8bs_dense_nt_mxfp4": [P] * 5 + [I] * 3 + [P],
        "fp8bs_grouped_contiguous_nt_mxfp4": [P] * 6 + [I] * 4 + [P],
        "fp8bs_grouped_masked_nt_mxfp4": [P] * 6 + [I] * 5 + [P],
        "fp8bs_gated_dense_mxfp4": [P] * 5 + [I] * 4 + [P],
        "fp8bs_gated_contiguous_mxfp4": [P] * 6 + [I] * 5 + [P],
        "fp8bs_gated_masked_mxfp4": [P] * 6 + [I] * 6 + [P],
        "fp8bs_gated_dense_mxfp4_q": [P] * 6 + [I] * 4 + [P],
        "fp8bs_gated_contiguous_mxfp4_q": [P] * 7 + [I] * 5 + [P],
        "fp8bs_gated_masked_mxfp4_q": [P] * 7 + [I] * 6 + [P],
        "fp8bs_gated_dense_mxfp4_backward": [P] * 7 + [I] * 6 + [P, S, P],
        "fp8bs_gated_contiguous_mxfp4_backward": [P] * 7 + [I] * 2 + [P] + [I] * 5 + [P, S, P],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = I
    lib.fp8bs_feed_forward_mxfp4.argtypes = [I, P, I] + [P] * 6 + [I] * 7 + [P, S, P]
    lib.fp8bs_feed_forward_mxfp4.restype = I
    lib.fp8bs_feed_forward_workspace_size.argtypes = [I, ctypes.c_int64] + [I] * 3
    lib.fp8bs_feed_forward_workspace_size.restype = ctypes.c_int64
    lib.fp8bs_gated_backward_workspace_size.argtypes = [I, ctypes.c_int64] + [I] * 5
    lib.fp8bs_gated_backward_workspace_size.restype = ctypes.c_int64
    _lib = lib
    return lib


# ---- argument checks ---------------------------------------------------------
# These run on every call of a decode step, so the common case -- contiguous tensors of the
# right type -- is a handful of attribute reads; _dev_ptr names what is wrong otherwise.

def _ptr(t, name, dtypes, ndim, index):
    """Address of a contiguous tensor of ndim dims on device `index`."""
    if (type(t) is _Tensor and t.is_cuda and t.dtype in dtypes and t.is_contiguous()
            and t.ndim == ndim):
        if t.get_device() == index:
            return t.data_ptr()
    else:
        p = _dev_ptr(t, name, dtypes, ndim)
        if t.get_device() == index:
            return p.value
    raise ValueError(f"{name} is on another device than the first operand")


def _scales(t, name, count, index):
    """Address of an exponent tensor of `count` words."""
    if type(t) is _Tensor and t.is_cuda and t.dtype is _i32 and t.is_contiguous():
        p = t.data_ptr()
    else:
        p = _dev_ptr(t, name, _INT32).value
    if t.numel() != count:
        raise ValueError(f"{name}: scale tensor sizes do not match the shapes")
    if t.get_device() != index:
        raise ValueError(f"{name} is on another device than the first operand")
    return p


def _ld(rows):
    return (rows + 3) & -4


def _first(t, name):
    """Device index of a call's first operand."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _call(name, index, stream, *args):
    """Calls the library on device `index` and the given (or its current) stream."""
    if index == _device_index():
        st = getattr(_lib, name)(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        torch = _torch()
        with torch.cuda.device(index):
            st = getattr(_lib, name)(*args, _raw_stream(index) if stream is None
                                     else stream.cuda_stream)
    if st:
        raise FP8BSError(st, name)


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}, expected one of {sorted(ACTIVATIONS)}")
    return code


def _operands(a, sfa, b, sfb, masked, grouped):
    """Device, checked addresses of A, its exponents, B and its exponents; rows of a slot, B
    rows, k, groups of B."""
    if _lib is None:
        _load()
    index = _first(a, "a")
    pa = _ptr(a, "a", _FP4, 3 if masked else 2, index)
    pb = _ptr(b, "b", _FP4, 3 if grouped else 2, index)
    sa, sb = a.shape, b.shape
    m, n, half = sa[-2], sb[-2], sa[-1]
    if sb[-1] != half:
        raise ValueError("shape mismatch between a and b")
    if half & 63 or not half or half > 1 << 23:
        raise FP8BSError(1, "k must be a positive multiple of 128, at most 2^24")
    groups = sb[0] if grouped else 1
    words = half // 64
    return (index, pa, _scales(sfa, "sfa", (sa[0] if masked else 1) * words * ((m + 3) & -4), index),
            pb, _scales(sfb, "sfb", groups * words * ((n + 3) & -4), index), m, n, 2 * half, groups)


def _rows_out(d, name, dtypes, a, cols, index):
    """Address of an output with a's rows and `cols` columns."""
    p = _ptr(d, name, dtypes, a.ndim, index)
    if d.shape[:-1] != a.shape[:-1] or d.shape[-1] != cols:
        raise ValueError(f"{name} must be {tuple(a.shape[:-1]) + (cols,)}, got {tuple(d.shape)}")
    return p


def _layout_data(layout, data, a, b, index):
    """Address of grouped_layout ("contiguous") or masked_m ("masked"), checked against a, b."""
    if layout == "contiguous":
        p = _ptr(data, "grouped_layout", _INT32, 1, index)
        if data.shape[0] != a.shape[0]:
            raise ValueError("grouped_layout must have one entry per row of a")
    else:
        p = _ptr(data, "masked_m", _INT32, 1, index)
        if b.shape[0] != a.shape[0] or data.shape[0] != a.shape[0]:
            raise ValueError("a, b and masked_m must have the same number of groups")
    return p


def _new(shape, dtype, index, stream):
    """Uninitialised device tensor, allocated for the stream it is used on."""
    if stream is None:
        return _empty(shape, dtype=dtype, device=index)
    with _torch().cuda.stream(stream):
        return _empty(shape, dtype=dtype, device=index)


# ---- quantiser ---------------------------------------------------------------

def _values(x, name):
    """(device, groups, rows, k) of a matrix of values or of codes."""
    if _lib is None:
        _load()
    index = _first(x, name)
    s = x.shape
    if s and s[-1] > 1 << 24:                  # (longer ones do not all fit the call's int)
        raise FP8BSError(1, "k must be a positive multiple of 128, at most 2^24")
    if len(s) == 2:
        return index, 1, s[0], s[1]
    if len(s) != 3:
        raise ValueError(f"{name} must be 2-D, or 3-D with groups")
    return index, s[0], s[1], s[2]


def fp8bs_quantize_mxfp4(x, q, sf, stream=None):
    """x bf16 or f32 [(groups,) rows, k] -> q codes [..., rows, k/2], sf int32 exponents
    [..., k/128, get_sfa_ld(rows)] (alignment padding not written)."""
    index, groups, rows, k = _values(x, "x")
    xp = _ptr(x, "x", _FLOAT, x.ndim, index)
    qp = _rows_out(q, "q", _FP4, x, k // 2, index)
    sp = _scales(sf, "sf", groups * (k // 128) * _ld(rows), index)
    _call("fp8bs_quantize_mxfp4", index, stream, xp, 1 if x.dtype is _bf16 else 0, qp, sp, groups,
          rows, k)


def fp8bs_dequantize_mxfp4(q, sf, x, stream=None):
    """The values that q and sf stand for, into x (bf16 or f32 [(groups,) rows, k])."""
    index, groups, rows, half = _values(q, "q")
    qp = _ptr(q, "q", _FP4, q.ndim, index)
    sp = _scales(sf, "sf", groups * (half // 64) * _ld(rows), index)
    xp = _rows_out(x, "x", _FLOAT, q, 2 * half, index)
    _call("fp8bs_dequantize_mxfp4", index, stream, qp, sp, xp, 1 if x.dtype is _bf16 else 0,
          groups, rows, 2 * half)


def quantize_mxfp4(x, stream=None):
    """(codes, exponents) of x; see ``fp8bs_quantize_mxfp4``."""
    index, groups, rows, k = _values(x, "x")
    xp = _ptr(x, "x", _FLOAT, x.ndim, index)
    lead = () if x.ndim == 2 else (groups,)
    q = _new((*lead, rows, k // 2), _u8, index, stream)
    sf = _new((*lead, k // 128, (rows + 3) & -4), _i32, index, stream)
    _call("fp8bs_quantize_mxfp4", index, stream, xp, 1 if x.dtype is _bf16 else 0, q.data_ptr(),
          sf.data_ptr(), groups, rows, k)
    return q, sf


def dequantize_mxfp4(q, sf, dtype=None, stream=None):
    """The values that q and sf stand for, bf16 (exact) unless dtype says float32."""
    index, groups, rows, half = _values(q, "q")
    qp = _ptr(q, "q", _FP4, q.ndim, index)
    sp = _scales(sf, "sf", groups * (half // 64) * ((rows + 3) & -4), index)
    if dtype is None:
        dtype = _bf16
    elif dtype not in _FLOAT:
        raise TypeError(f"dtype must be one of {_FLOAT}")
    x = _new((*q.shape[:-1], 2 * half), dtype, index, stream)
    _call("fp8bs_dequantize_mxfp4", index, stream, qp, sp, x.data_ptr(),
          1 if dtype is _bf16 else 0, groups, rows, 2 * half)
    return x


# ---- product -----------------------------------------------------------------

def fp8bs_dense_nt_mxfp4(a, sfa, b, sfb, d, stream=None):
    """D = A B^T: a codes [m][k/2], b codes [n][k/2], d bf16 [m][n] (written)."""
    index, pa, psa, pb, psb, m, n, k, _ = _operands(a, sfa, b, sfb, False, False)
    dp = _rows_out(d, "d", _BF16, a, n, index)
    _call("fp8bs_dense_nt_mxfp4", index, stream, pa, psa, pb, psb, dp, m, n, k)


def fp8bs_grouped_contiguous_nt_mxfp4(a, sfa, b, sfb, d, grouped_layout, stream=None):
    """Contiguous MoE layout: a [m_total][k/2], b [g][n][k/2], grouped_layout int32 [m_total]."""
    index, pa, psa, pb, psb, m, n, k, g = _operands(a, sfa, b, sfb, False, True)
    lp = _layout_data("contiguous", grouped_layout, a, b, index)
    dp = _rows_out(d, "d", _BF16, a, n, index)
    _call("fp8bs_grouped_contiguous_nt_mxfp4", index, stream, pa, psa, pb, psb, dp, lp, m, n, k, g)


def fp8bs_grouped_masked_nt_mxfp4(a, sfa, b, sfb, d, masked_m, expected_m: int = 0, stream=None):
    """Masked MoE layout: a [g][max_m][k/2], b [g][n][k/2], d bf16 [g][max_m][n]."""
    index, pa, psa, pb, psb, m, n, k, g = _operands(a, sfa, b, sfb, True, True)
    mp = _layout_data("masked", masked_m, a, b, index)
    dp = _rows_out(d, "d", _BF16, a, n, index)
    _call("fp8bs_grouped_masked_nt_mxfp4", index, stream, pa, psa, pb, psb, dp, mp, g, m,
          int(expected_m), n, k)


# ---- gated block -------------------------------------------------------------

def _gated(layout, a, sfa, b, sfb, out, data, expected_m, activation, stream):
    """out: (h,) or (hq, sfh)."""
    grouped, masked = layout != "dense", layout == "masked"
    index, pa, psa, pb, psb, m, n, k, g = _operands(a, sfa, b, sfb, masked, grouped)
    act = _activation(activation)
    if n % 2:
        raise ValueError("b must hold 2f rows")
    f = n // 2
    if len(out) == 2:
        name = f"fp8bs_gated_{layout}_mxfp4_q"
        outs = (_rows_out(out[0], "hq", _FP4, a, f // 2, index),
                _scales(out[1], "sfh", (a.shape[0] if masked else 1) * (f // 128) * _ld(m), index))
    else:
        name = f"fp8bs_gated_{layout}_mxfp4"
        outs = (_rows_out(out[0], "h", _BF16, a, f, index),)
    if not grouped:
        _call(name, index, stream, pa, psa, pb, psb, *outs, m, f, k, act)
        return
    p = _layout_data(layout, data, a, b, index)
    if masked:
        _call(name, index, stream, pa, psa, pb, psb, *outs, p, g, m, int(expected_m), f, k, act)
    else:
        _call(name, index, stream, pa, psa, pb, psb, *outs, p, m, f, k, g, act)


def fp8bs_gated_dense_mxfp4(a, sfa, b, sfb, h, activation: str = "silu", stream=None):
    """h = act(A Wg^T) * (A Wu^T): a codes [m][k/2], b codes [2f][k/2] (gate rows, then up
    rows), h bf16 [m][f] (written)."""
    _gated("dense", a, sfa, b, sfb, (h,), None, 0, activation, stream)


def fp8bs_gated_contiguous_mxfp4(a, sfa, b, sfb, h, grouped_layout, activation: str = "silu",
                                 stream=None):
    """Contiguous MoE layout of the gated block: b [g][2f][k/2], h bf16 [m_total][f]."""
    _gated("contiguous", a, sfa, b, sfb, (h,), grouped_layout, 0, activation, stream)


def fp8bs_gated_masked_mxfp4(a, sfa, b, sfb, h, masked_m, expected_m: int = 0,
                             activation: str = "silu", stream=None):
    """Masked MoE layout of the gated block: a [g][max_m][k/2], h bf16 [g][max_m][f]."""
    _gated("masked", a, sfa, b, sfb, (h,), masked_m, expected_m, activation, stream)


def fp8bs_gated_dense_mxfp4_q(a, sfa, b, sfb, hq, sfh, activation: str = "silu", stream=None):
    """The gated block with h quantised: hq codes [m][f/2], sfh int32 [f/128][get_sfa_ld(m)]."""
    _gated("dense", a, sfa, b, sfb, (hq, sfh), None, 0, activation, stream)


def fp8bs_gated_contiguous_mxfp4_q(a, sfa, b, sfb, hq, sfh, grouped_layout,
                                   activation: str = "silu", stream=None):
    """fp8bs_gated_contiguous_mxfp4 with h quantised."""
    _gated("contiguous", a, sfa, b, sfb, (hq, sfh), grouped_layout, 0, activation, stream)


def fp8bs_gated_masked_mxfp4_q(a, sfa, b, sfb, hq, sfh, masked_m, expected_m: int = 0,
                               activation: str = "silu", stream=None):
    """fp8bs_gated_masked_mxfp4 with h quantised (sfh [g][f/128][get_sfa_ld(max_m)])."""
    _gated("masked", a, sfa, b, sfb, (hq, sfh), masked_m, expected_m, activation, stream)


# ---- backward ----------------------------------------------------------------

def gated_backward_workspace_size(layout: int, m: int, f: int, k: int, num_groups: int = 1,
                                  want_da: bool = True, want_db: bool = True) -> int:
    """Workspace bytes of the backward pass (layout: LAYOUT_DENSE or LAYOUT_CONTIGUOUS)."""
    v = int(_load().fp8bs_gated_backward_workspace_size(int(layout), int(m), int(f), int(k),
                                                        int(num_groups), int(bool(want_da)),
                                                        int(bool(want_db))))
    if v < 0:
        raise FP8BSError(-v, "fp8bs_gated_backward_workspace_size")
    return v


def _workspace(workspace, size, index, stream):
    """(address, bytes, tensor) of the caller's workspace, or of a new one of size() bytes."""
    if workspace is None:
        workspace = _new((size(),), _u8, index, stream)
    return _ptr(workspace, "workspace", _UINT8, 1, index), workspace.shape[0], workspace


def _backward(layout, a, sfa, b, sfb, dh, da, db, data, activation, accumulate, workspace, stream):
    grouped = layout == "contiguous"
    index, pa, psa, pb, psb, m, n, k, g = _operands(a, sfa, b, sfb, False, grouped)
    act = _activation(activation)
    if n % 2:
        raise ValueError("b must hold 2f rows")
    f = n // 2
    dhp = _rows_out(dh, "dh", _BF16, a, f, index)
    dap = None if da is None else _rows_out(da, "da", _BF16, a, k, index)
    dbp, f32 = None, False
    if db is not None:
        dbp = _rows_out(db, "db", _FLOAT, b, k, index)
        f32 = db.dtype is _f32
    if accumulate and not f32:
        raise ValueError("accumulate needs a float32 db")
    wp, wb, _keep = _workspace(
        workspace, lambda: gated_backward_workspace_size(
            LAYOUT_CONTIGUOUS if grouped else LAYOUT_DENSE, m, f, k, g, da is not None,
            db is not None), index, stream)
    head = (pa, psa, pb, psb, dhp, dap, dbp, 0 if f32 else 1, 1 if accumulate else 0)
    if grouped:
        p = _layout_data(layout, data, a, b, index)
        _call("fp8bs_gated_contiguous_mxfp4_backward", index, stream, *head, p, m, f, k, g, act, wp,
              wb)
    else:
        _call("fp8bs_gated_dense_mxfp4_backward", index, stream, *head, m, f, k, act, wp, wb)


def fp8bs_gated_dense_mxfp4_backward(a, sfa, b, sfb, dh, da, db, activation: str = "silu",
                                     accumulate: bool = False, workspace=None, stream=None):
    """Gradients of the gated block with respect to the values a and b stand for: dh bf16
    [m][f] -> da bf16 [m][k], db bf16 or f32 [2f][k]; either may be None.  accumulate adds to
    an f32 db.  workspace: uint8 tensor of gated_backward_workspace_size() bytes, or None to
    allocate one."""
    _backward("dense", a, sfa, b, sfb, dh, da, db, None, activation, accumulate, workspace, stream)


def fp8bs_gated_contiguous_mxfp4_backward(a, sfa, b, sfb, dh, da, db, grouped_layout,
                                          activation: str = "silu", accumulate: bool = False,
                                          workspace=None, stream=None):
    """Contiguous MoE layout of the backward pass: db [g][2f][k]; da written at valid rows."""
    _backward("contiguous", a, sfa, b, sfb, dh, da, db, grouped_layout, activation, accumulate,
              workspace, stream)


# ---- a feed-forward layer ----------------------------------------------------

def feed_forward_workspace_size(layout: int, m: int, f: int, k: int, num_groups: int = 1) -> int:
    """Workspace bytes of ``fp8bs_feed_forward_mxfp4`` (m: rows, of a slot if masked)."""
    v = int(_load().fp8bs_feed_forward_workspace_size(int(layout), int(m), int(f), int(k),
                                                      int(num_groups)))
    if v < 0:
        raise FP8BSError(-v, "fp8bs_feed_forward_workspace_size")
    return v


def fp8bs_feed_forward_mxfp4(x, b, sfb, b2, sfb2, out, activation: str = "silu",
                             grouped_layout=None, masked_m=None, expected_m: int = 0,
                             workspace=None, stream=None):
    """out = MXFP4(act(x Wg^T) * (x Wu^T)) W2^T with x quantised to MXFP4.

    x bf16 or f32 [m][k] (masked: [g][max_m][k]); b codes [(g,) 2f, k/2] of the gate and up
    projections, b2 codes [(g,) n, f/2] of the down projection; out bf16 [.., n].
    grouped_layout or masked_m select the MoE layouts.  workspace: uint8 tensor of
    feed_forward_workspace_size() bytes, or None to allocate one."""
    if grouped_layout is not None and masked_m is not None:
        raise ValueError("grouped_layout and masked_m exclude each other")
    index, slots, m, k = _values(x, "x")
    masked, grouped = masked_m is not None, masked_m is not None or grouped_layout is not None
    xp = _ptr(x, "x", _FLOAT, 3 if masked else 2, index)
    pb = _ptr(b, "b", _FP4, 3 if grouped else 2, index)
    pb2 = _ptr(b2, "b2", _FP4, 3 if grouped else 2, index)
    groups = b.shape[0] if grouped else 1
    two_f, n = b.shape[-2], b2.shape[-2]
    f = two_f // 2
    if 2 * b.shape[-1] != k or two_f % 2 or 2 * b2.shape[-1] != f or (
            grouped and b2.shape[0] != groups):
        raise ValueError("shape mismatch between x, b and b2")
    psb = _scales(sfb, "sfb", groups * (k // 128) * _ld(two_f), index)
    psb2 = _scales(sfb2, "sfb2", groups * (f // 128) * _ld(n), index)
    act = _activation(activation)
    op = _rows_out(out, "out", _BF16, x, n, index)
    code, data = LAYOUT_DENSE, None
    if masked:
        code, data = LAYOUT_MASKED, _layout_data("masked", masked_m, x, b, index)
    elif grouped:
        code, data = LAYOUT_CONTIGUOUS, _layout_data("contiguous", grouped_layout, x, b, index)
    wp, wb, _keep = _workspace(workspace,
                               lambda: feed_forward_workspace_size(code, m, f, k, groups), index,
                               stream)
    _call("fp8bs_feed_forward_mxfp4", index, stream, code, xp, 1 if x.dtype is _bf16 else 0, pb, psb,
          pb2, psb2, op, data, m, int(expected_m), f, k, n, groups, act, wp, wb)


def feed_forward_mxfp4(x, b, sfb, b2, sfb2, activation: str = "silu", out=None,
                       grouped_layout=None, masked_m=None, expected_m: int = 0, stream=None):
    """``fp8bs_feed_forward_mxfp4`` that returns its output, a new tensor unless given (rows
    that are not valid are not written)."""
    if out is None:
        index, _, _, _ = _values(x, "x")
        out = _new((*x.shape[:-1], b2.shape[-2]), _bf16, index, stream)
    fp8bs_feed_forward_mxfp4(x, b, sfb, b2, sfb2, out, activation, grouped_layout, masked_m,
                             expected_m, None, stream)
    return out
