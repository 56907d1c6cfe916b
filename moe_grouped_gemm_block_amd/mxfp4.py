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
from moe_grouped_gemm_block_amd import (FP8BSError, LAYOUT_CONTIGUOUS, LAYOUT_DENSE, _bf16_dtypes,
                                        _check, _dev_ptr, _DTYPES, _on_device,
                                        _stream_handle, _torch, get_sfa_ld)

__all__ = [
    "fp8bs_quantize_mxfp4", "fp8bs_dequantize_mxfp4", "quantize_mxfp4", "dequantize_mxfp4",
    "fp8bs_dense_nt_mxfp4", "fp8bs_grouped_contiguous_nt_mxfp4", "fp8bs_grouped_masked_nt_mxfp4",
    "fp8bs_gated_dense_mxfp4", "fp8bs_gated_contiguous_mxfp4", "fp8bs_gated_masked_mxfp4",
    "fp8bs_gated_dense_mxfp4_q", "fp8bs_gated_contiguous_mxfp4_q", "fp8bs_gated_masked_mxfp4_q",
    "fp8bs_gated_dense_mxfp4_backward", "fp8bs_gated_contiguous_mxfp4_backward",
    "gated_backward_workspace_size", "feed_forward_mxfp4", "ACTIVATIONS",
]

ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}

_NULL = ctypes.c_void_p(None)
_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    lib = _pkg._load()
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
    lib.fp8bs_gated_backward_workspace_size.argtypes = [I, ctypes.c_int64] + [I] * 5
    lib.fp8bs_gated_backward_workspace_size.restype = ctypes.c_int64
    _lib = lib
    return lib


# ---- argument checks ---------------------------------------------------------

def _fp4_dtypes():
    d = _DTYPES.get("fp4")
    if d is None:
        torch = _torch()
        d = (torch.uint8,)
        packed = getattr(torch, "float4_e2m1fn_x2", None)
        if packed is not None:
            d += (packed,)
        _DTYPES["fp4"] = d
    return d


def _float_dtypes():
    d = _DTYPES.get("float")
    if d is None:
        torch = _torch()
        d = _DTYPES["float"] = (torch.bfloat16, torch.float32)
    return d


def _int32():
    d = _DTYPES.get("int32")
    if d is None:
        d = _DTYPES["int32"] = (_torch().int32,)
    return d


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}, expected one of {sorted(ACTIVATIONS)}")
    return code


def _same_device(*tensors):
    index = tensors[0].get_device()
    for t in tensors[1:]:
        if t.get_device() != index:
            raise ValueError("all tensors must be on one device")


def _operands(a, sfa, b, sfb, a_ndim, b_ndim):
    """Checked pointers of A, its exponents, B and its exponents; (rows of a slot, B rows, k,
    groups of B)."""
    ptrs = (_dev_ptr(a, "a", _fp4_dtypes(), a_ndim), _dev_ptr(sfa, "sfa", _int32()),
            _dev_ptr(b, "b", _fp4_dtypes(), b_ndim), _dev_ptr(sfb, "sfb", _int32()))
    m, k = a.shape[-2], 2 * a.shape[-1]
    n, groups = b.shape[-2], b.shape[0] if b_ndim == 3 else 1
    if 2 * b.shape[-1] != k:
        raise ValueError("shape mismatch between a and b")
    if k % 128 == 0:
        kw = k // 128
        slots = a.shape[0] if a_ndim == 3 else 1
        if (sfa.numel() != slots * kw * get_sfa_ld(m)
                or sfb.numel() != groups * kw * get_sfa_ld(n)):
            raise ValueError("scale tensor sizes do not match the shapes")
    return ptrs, m, n, k, groups


def _layout_data(layout, data, a, b):
    """Pointer of grouped_layout ("contiguous") or masked_m ("masked"), checked against a, b."""
    if layout == "contiguous":
        p = _dev_ptr(data, "grouped_layout", _int32(), 1)
        if data.shape[0] != a.shape[0]:
            raise ValueError("grouped_layout must have one entry per row of a")
    else:
        p = _dev_ptr(data, "masked_m", _int32(), 1)
        if b.shape[0] != a.shape[0] or data.shape[0] != a.shape[0]:
            raise ValueError("a, b and masked_m must have the same number of groups")
    return p


# ---- quantiser ---------------------------------------------------------------

def _quant_shape(x, q, sf):
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows][k] or [groups][rows][k]")
    rows, k = x.shape[-2], x.shape[-1]
    groups = x.shape[0] if x.dim() == 3 else 1
    if tuple(q.shape) != tuple(x.shape[:-1]) + (k // 2,):
        raise ValueError("q must be [..., rows, k/2] of x")
    if k % 128 == 0 and sf.numel() != groups * (k // 128) * get_sfa_ld(rows):
        raise ValueError("sf must be [..., k/128, get_sfa_ld(rows)]")
    _same_device(x, q, sf)
    return groups, rows, k


def fp8bs_quantize_mxfp4(x, q, sf, stream=None):
    """x bf16 or f32 [(groups,) rows, k] -> q codes [..., rows, k/2], sf int32 exponents
    [..., k/128, get_sfa_ld(rows)] (alignment padding not written)."""
    groups, rows, k = _quant_shape(x, q, sf)
    xp = _dev_ptr(x, "x", _float_dtypes())
    args = (_dev_ptr(q, "q", _fp4_dtypes()), _dev_ptr(sf, "sf", _int32()))
    dtype = 1 if x.dtype == _torch().bfloat16 else 0
    with _on_device(x):
        st = _load().fp8bs_quantize_mxfp4(xp, dtype, *args, groups, rows, k,
                                          _stream_handle(stream, x.device))
    _check(st, "fp8bs_quantize_mxfp4")


def fp8bs_dequantize_mxfp4(q, sf, x, stream=None):
    """The values that q and sf stand for, into x (bf16 or f32 [(groups,) rows, k])."""
    groups, rows, k = _quant_shape(x, q, sf)
    args = (_dev_ptr(q, "q", _fp4_dtypes()), _dev_ptr(sf, "sf", _int32()))
    xp = _dev_ptr(x, "x", _float_dtypes())
    dtype = 1 if x.dtype == _torch().bfloat16 else 0
    with _on_device(x):
        st = _load().fp8bs_dequantize_mxfp4(*args, xp, dtype, groups, rows, k,
                                            _stream_handle(stream, x.device))
    _check(st, "fp8bs_dequantize_mxfp4")


def _empty(shape, dtype, like, stream):
    """Uninitialised tensor on like's device, allocated for the stream it is used on."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def quantize_mxfp4(x, stream=None):
    """(codes, exponents) of x; see ``fp8bs_quantize_mxfp4``."""
    torch = _torch()
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows][k] or [groups][rows][k]")
    lead, (rows, k) = tuple(x.shape[:-2]), x.shape[-2:]
    q = _empty(lead + (rows, k // 2), torch.uint8, x, stream)
    sf = _empty(lead + (k // 128, get_sfa_ld(rows)), torch.int32, x, stream)
    fp8bs_quantize_mxfp4(x, q, sf, stream)
    return q, sf


def dequantize_mxfp4(q, sf, dtype=None, stream=None):
    """The values that q and sf stand for, bf16 (exact) unless dtype says float32."""
    torch = _torch()
    x = _empty(tuple(q.shape[:-1]) + (2 * q.shape[-1],), dtype or torch.bfloat16, q, stream)
    fp8bs_dequantize_mxfp4(q, sf, x, stream)
    return x


# ---- product -----------------------------------------------------------------

def _rows_out(d, name, a, cols):
    if tuple(d.shape) != tuple(a.shape[:-1]) + (cols,):
        raise ValueError(f"{name} must be {tuple(a.shape[:-1]) + (cols,)}, got {tuple(d.shape)}")


def fp8bs_dense_nt_mxfp4(a, sfa, b, sfb, d, stream=None):
    """D = A B^T: a codes [m][k/2], b codes [n][k/2], d bf16 [m][n] (written)."""
    ptrs, m, n, k, _ = _operands(a, sfa, b, sfb, 2, 2)
    dp = _dev_ptr(d, "d", _bf16_dtypes(), 2)
    _rows_out(d, "d", a, n)
    _same_device(a, sfa, b, sfb, d)
    with _on_device(a):
        st = _load().fp8bs_dense_nt_mxfp4(*ptrs, dp, m, n, k, _stream_handle(stream, a.device))
    _check(st, "fp8bs_dense_nt_mxfp4")


def fp8bs_grouped_contiguous_nt_mxfp4(a, sfa, b, sfb, d, grouped_layout, stream=None):
    """Contiguous MoE layout: a [m_total][k/2], b [g][n][k/2], grouped_layout int32 [m_total]."""
    ptrs, m, n, k, g = _operands(a, sfa, b, sfb, 2, 3)
    lp = _layout_data("contiguous", grouped_layout, a, b)
    dp = _dev_ptr(d, "d", _bf16_dtypes(), 2)
    _rows_out(d, "d", a, n)
    _same_device(a, sfa, b, sfb, d, grouped_layout)
    with _on_device(a):
        st = _load().fp8bs_grouped_contiguous_nt_mxfp4(*ptrs, dp, lp, m, n, k, g,
                                                       _stream_handle(stream, a.device))
    _check(st, "fp8bs_grouped_contiguous_nt_mxfp4")


def fp8bs_grouped_masked_nt_mxfp4(a, sfa, b, sfb, d, masked_m, expected_m: int = 0, stream=None):
    """Masked MoE layout: a [g][max_m][k/2], b [g][n][k/2], d bf16 [g][max_m][n]."""
    ptrs, m, n, k, g = _operands(a, sfa, b, sfb, 3, 3)
    mp = _layout_data("masked", masked_m, a, b)
    dp = _dev_ptr(d, "d", _bf16_dtypes(), 3)
    _rows_out(d, "d", a, n)
    _same_device(a, sfa, b, sfb, d, masked_m)
    with _on_device(a):
        st = _load().fp8bs_grouped_masked_nt_mxfp4(*ptrs, dp, mp, g, m, int(expected_m), n, k,
                                                   _stream_handle(stream, a.device))
    _check(st, "fp8bs_grouped_masked_nt_mxfp4")


# ---- gated block -------------------------------------------------------------

def _gated(layout, a, sfa, b, sfb, out, data, expected_m, activation, stream):
    """out: (h,) or (hq, sfh)."""
    quantised = len(out) == 2
    grouped = layout != "dense"
    ptrs, m, n, k, g = _operands(a, sfa, b, sfb, 3 if layout == "masked" else 2,
                                 3 if grouped else 2)
    act = _activation(activation)
    if n % 2:
        raise ValueError("b must hold 2f rows")
    f = n // 2
    if quantised:
        hq, sfh = out
        outs = (_dev_ptr(hq, "hq", _fp4_dtypes()), _dev_ptr(sfh, "sfh", _int32()))
        _rows_out(hq, "hq", a, f // 2)
        slots = a.shape[0] if layout == "masked" else 1
        if f % 128 == 0 and sfh.numel() != slots * (f // 128) * get_sfa_ld(m):
            raise ValueError("sfh must be [..., f/128, get_sfa_ld(rows)]")
    else:
        outs = (_dev_ptr(out[0], "h", _bf16_dtypes()),)
        _rows_out(out[0], "h", a, f)
    extra = (_layout_data(layout, data, a, b),) if grouped else ()
    _same_device(a, sfa, b, sfb, *out, *((data,) if grouped else ()))
    sizes = {"dense": (m, f, k), "contiguous": (m, f, k, g),
             "masked": (g, m, int(expected_m), f, k)}[layout]
    name = f"fp8bs_gated_{layout}_mxfp4" + ("_q" if quantised else "")
    with _on_device(a):
        st = getattr(_load(), name)(*ptrs, *outs, *extra, *sizes, act,
                                    _stream_handle(stream, a.device))
    _check(st, name)


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


def _backward(layout, a, sfa, b, sfb, dh, da, db, data, activation, accumulate, workspace, stream):
    torch = _torch()
    grouped = layout == "contiguous"
    ptrs, m, n, k, g = _operands(a, sfa, b, sfb, 2, 3 if grouped else 2)
    act = _activation(activation)
    if n % 2:
        raise ValueError("b must hold 2f rows")
    f = n // 2
    dhp = _dev_ptr(dh, "dh", _bf16_dtypes(), 2)
    _rows_out(dh, "dh", a, f)
    tensors = [a, sfa, b, sfb, dh]
    dap = dbp = _NULL
    f32 = False
    if da is not None:
        dap = _dev_ptr(da, "da", _bf16_dtypes(), 2)
        _rows_out(da, "da", a, k)
        tensors.append(da)
    if db is not None:
        dbp = _dev_ptr(db, "db", _float_dtypes(), b.dim())
        if tuple(db.shape) != tuple(b.shape[:-1]) + (k,):
            raise ValueError("db must have b's shape with k columns")
        f32 = db.dtype == torch.float32
        tensors.append(db)
    if accumulate and not f32:
        raise ValueError("accumulate needs a float32 db")
    extra = ()
    if grouped:
        extra = (_layout_data(layout, data, a, b),)
        tensors.append(data)
    _same_device(*tensors)
    sizes = (m, f, k, g) if grouped else (m, f, k)
    name = f"fp8bs_gated_{layout}_mxfp4_backward"
    with _on_device(a):
        if workspace is None:
            size = gated_backward_workspace_size(LAYOUT_CONTIGUOUS if grouped else LAYOUT_DENSE, m,
                                                 f, k, g, da is not None, db is not None)
            workspace = _empty((size,), torch.uint8, a, stream)
        wp = _dev_ptr(workspace, "workspace", (torch.uint8,), 1)
        _same_device(a, workspace)
        st = getattr(_load(), name)(*ptrs, dhp, dap, dbp, 0 if f32 else 1, int(bool(accumulate)),
                                    *extra, *sizes, act, wp, workspace.numel(),
                                    _stream_handle(stream, a.device))
    _check(st, name)


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

def feed_forward_mxfp4(x, b, sfb, b2, sfb2, activation: str = "silu", out=None,
                       grouped_layout=None, masked_m=None, expected_m: int = 0, stream=None):
    """y = MXFP4(act(x Wg^T) * (x Wu^T)) W2^T with x quantised to MXFP4.

    x bf16 or f32 [m][k] (masked: [g][max_m][k]); b codes [(g,) 2f, k/2] of the gate and up
    projections, b2 codes [(g,) n, f/2] of the down projection.  grouped_layout or masked_m
    select the MoE layouts.  Three launches: quantiser, gated block (h quantised in its
    epilogue), product.  out: bf16, allocated if None (rows that are not valid are not
    written)."""
    torch = _torch()
    if grouped_layout is not None and masked_m is not None:
        raise ValueError("grouped_layout and masked_m exclude each other")
    q, sf = quantize_mxfp4(x, stream)
    lead, m = tuple(x.shape[:-2]), x.shape[-2]
    f, n = b.shape[-2] // 2, b2.shape[-2]
    hq = _empty(lead + (m, f // 2), torch.uint8, x, stream)
    sfh = _empty(lead + (f // 128, get_sfa_ld(m)), torch.int32, x, stream)
    if out is None:
        out = _empty(lead + (m, n), torch.bfloat16, x, stream)
    if grouped_layout is not None:
        fp8bs_gated_contiguous_mxfp4_q(q, sf, b, sfb, hq, sfh, grouped_layout, activation, stream)
        fp8bs_grouped_contiguous_nt_mxfp4(hq, sfh, b2, sfb2, out, grouped_layout, stream)
    elif masked_m is not None:
        fp8bs_gated_masked_mxfp4_q(q, sf, b, sfb, hq, sfh, masked_m, expected_m, activation,
                                   stream)
        fp8bs_grouped_masked_nt_mxfp4(hq, sfh, b2, sfb2, out, masked_m, expected_m, stream)
    else:
        fp8bs_gated_dense_mxfp4_q(q, sf, b, sfb, hq, sfh, activation, stream)
        fp8bs_dense_nt_mxfp4(hq, sfh, b2, sfb2, out, stream)
    return out
