"""What stands between the products of an FP8 mixture-of-experts layer: the norm with e4m3
output, dispatch of tokens to their experts' rows and the weighted way back, the gated activation
with its e4m3 checkpoint, the quantiser along tokens for weight gradients -- and their backward
passes.

Binding of the calls that ``include/fp8bs.h`` describes under "Between the products"; argument
checks and marshalling only.  Operands in e4m3 are pairs of codes, uint8 (or
``torch.float8_e4m3fn``), and scales, float32: 1x128 as ``quantize_1x128`` gives them, 128x1 as
``fp8bs_k_grouped_tn_contiguous`` reads them.  Outputs are written in place; ``rms_norm_1x128``,
``moe_dispatch`` and ``quantize_128x1`` allocate what they return.

Each call goes first to the compiled module ``fp8bs_layer_py``, which looks the operands over and
calls the library; what it does not take -- a wrong operand, another device than the current one,
a workspace to allocate for another stream -- comes back here, to be named or done.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
from collections import namedtuple

import moe_grouped_gemm_block_amd as _pkg
from moe_grouped_gemm_block_amd import (DTYPE_BF16, DTYPE_F32, FP8BSError, LAYOUT_CONTIGUOUS,
                                        LAYOUT_DENSE, LAYOUT_MASKED, _torch)
from moe_grouped_gemm_block_amd import mxfp4 as _mx
from moe_grouped_gemm_block_amd.mxfp4 import _activation, _call, _first, _new, _ptr

__all__ = [
    "fp8bs_rms_norm", "fp8bs_rms_norm_backward", "rms_norm_backward_workspace_size",
    "rms_norm_1x128", "fp8bs_moe_dispatch", "moe_dispatch", "moe_capacity",
    "moe_dispatch_workspace_size", "Dispatched", "fp8bs_moe_combine", "fp8bs_moe_combine_backward",
    "fp8bs_gated_quantize", "fp8bs_gated_quantize_backward", "fp8bs_quantize_128x1",
    "quantize_128x1", "DTYPE_E4M3",
]

DTYPE_E4M3 = 2

_lib = None
_quick = None                                       # the compiled module, once the library is loaded
_MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "fp8bs_layer_py.so")


def _load_module(lib):
    if not os.path.exists(_MODULE_PATH):
        raise RuntimeError(f"{_MODULE_PATH} is missing; build it with "
                           "`python -m moe_grouped_gemm_block_amd.build`")
    spec = importlib.util.spec_from_file_location("fp8bs_layer_py", _MODULE_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.use(*(ctypes.cast(getattr(lib, "fp8bs_" + name), ctypes.c_void_p).value for name in (
        "rms_norm", "rms_norm_backward_workspace_size", "rms_norm_backward",
        "moe_dispatch_workspace_size", "moe_dispatch", "moe_combine", "moe_combine_backward",
        "gated_quantize", "gated_quantize_backward", "quantize_128x1")),
        _mx._raw_stream)
    return module


def _done(status, name):
    """Whether the compiled module made the call (it answers -1 if not)."""
    if status > 0:
        raise FP8BSError(status, name)
    return status == 0


def _number(stream):
    return None if stream is None else stream.cuda_stream


def _load():
    """The library with this module's prototypes."""
    global _lib, _quick, _Tensor, _FP8, _BF16, _F32, _FLOAT, _INT32, _IDS, _KEPT, _ROWS, _CODE, _bf16, _u8, _f32
    if _lib is not None:
        return _lib
    lib = _mx._load()
    torch = _torch()
    _Tensor = torch.Tensor
    _bf16, _u8, _f32 = torch.bfloat16, torch.uint8, torch.float32
    _FP8, _BF16, _F32 = _pkg._fp8_dtypes(), _pkg._bf16_dtypes(), (torch.float32,)
    _FLOAT, _INT32, _IDS = (_bf16, _f32), (torch.int32,), (torch.int32, torch.int64)
    _KEPT = (*_FP8, _bf16)                          # a checkpoint, or the values themselves
    _ROWS = (*_FP8, _bf16, _f32)
    _CODE = {_bf16: DTYPE_BF16, _f32: DTYPE_F32, **{t: DTYPE_E4M3 for t in _FP8}}
    P, I, I64, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    for name, args in {
        "fp8bs_rms_norm": [P, I, P, P, I, P, I, P, I, P, P, P, I, I, ctypes.c_float, P],
        "fp8bs_rms_norm_backward": [P, I, P, P, I, P, I, P, P, P, I, I, I, P, S, P],
        "fp8bs_moe_dispatch": [I, P, I, P, I] + [P] * 6 + [I] * 5 + [P, S, P],
        "fp8bs_moe_combine": [P] * 4 + [I, I64, I, I, I, P],
        "fp8bs_moe_combine_backward": [P, I] + [P] * 7 + [I] * 5 + [P],
        "fp8bs_gated_quantize": [I] + [P] * 6 + [I] * 4 + [P],
        "fp8bs_gated_quantize_backward": [P, I] + [P] * 10 + [I] * 3 + [P],
        "fp8bs_quantize_128x1": [P, I, P, P, P, P, I, I, P],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = I
    lib.fp8bs_rms_norm_backward_workspace_size.argtypes = [I64, I]
    lib.fp8bs_moe_capacity.argtypes = [I64, I, I]
    lib.fp8bs_moe_dispatch_workspace_size.argtypes = [I, I64, I, I, I64]
    for name in ("fp8bs_rms_norm_backward_workspace_size", "fp8bs_moe_capacity",
                 "fp8bs_moe_dispatch_workspace_size"):
        getattr(lib, name).restype = I64
    _quick = _load_module(lib)
    _lib = lib
    return lib


# ---- argument checks -----------------------------------------------------------

# These run on every call of a decode step: the common case -- contiguous tensors of the right type
# and shape on the device -- is a few attribute reads; _ptr names what is wrong otherwise.

def _start(t, name):
    """Device index of a call's first operand."""
    if _lib is None:
        _load()
    if type(t) is _Tensor:
        index = t.get_device()
        if index >= 0:
            return index
    return _first(t, name)


def _like(t, name, dtypes, shape, index):
    """Address of a tensor of a given shape."""
    if (isinstance(t, _Tensor) and t.dtype in dtypes and t.get_device() == index and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    p = _ptr(t, name, dtypes, len(shape), index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return p


def _scales(t, name, count, index):
    """Address of `count` float32 scales."""
    if (isinstance(t, _Tensor) and t.dtype is _f32 and t.get_device() == index
            and t.numel() == count and t.is_contiguous()):
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name} is missing: codes come with their scales")
    p = _ptr(t, name, _F32, t.ndim if isinstance(t, _Tensor) else 0, index)
    if t.numel() != count:
        raise ValueError(f"{name}: scale tensor sizes do not match the shapes")
    return p


def _ld(rows):
    return (rows + 3) & -4


def _codes(q, sf, names, slots, rows, k, shape, index):
    """Addresses of an optional 1x128 output."""
    if q is None:
        if sf is not None:
            raise ValueError(f"{names[1]} without {names[0]}")
        return None, None
    qp = _like(q, names[0], _FP8, shape, index)
    return qp, _scales(sf, names[1], slots * (k // 128) * _ld(rows), index)


def _columns(q, sf, names, rows, n, index):
    """Addresses of an optional 128x1 output."""
    if q is None:
        if sf is not None:
            raise ValueError(f"{names[1]} without {names[0]}")
        return None, None
    padded = (rows + 127) // 128 * 128
    qp = _like(q, names[0], _FP8, (padded, n), index)
    return qp, _scales(sf, names[1], padded // 128 * _ld(n), index)


def _size(name, *args):
    v = int(getattr(_load(), name)(*(int(a) for a in args)))
    if v < 0:
        raise FP8BSError(-v, name)
    return v


def _space(workspace, size, index, stream):
    """(address, bytes, tensor) of the caller's workspace, or of a new one of size() bytes."""
    if workspace is None:
        n = size()
        if n == 0:
            return None, 0, None
        workspace = _new((n,), _u8, index, stream)
    return _ptr(workspace, "workspace", (_u8,), 1, index), workspace.shape[0], workspace


_MOST = 0x7FFFFFFF                                  # (the calls take sizes as int: more would wrap)


def _within(name, *sizes):
    for n in sizes:
        if n > _MOST:
            raise FP8BSError(1, f"{name}: sizes are at most 2^31 - 1")


def _matrix(t, name, dtypes, index):
    """(address, rows, columns) of a matrix."""
    if not (isinstance(t, _Tensor) and t.dtype in dtypes and t.get_device() == index
            and t.ndim == 2 and t.is_contiguous()):
        _ptr(t, name, dtypes, 2, index)
    rows, columns = t.shape
    if columns > 1 << 24 or rows > _MOST:
        raise FP8BSError(1, f"{name}: at most 2^24 columns and 2^31 - 1 rows")
    return t.data_ptr(), rows, columns


# ---- norm ------------------------------------------------------------------------

def fp8bs_rms_norm(x, weight, residual=None, residual_out=None, y=None, q=None, sfa=None,
                   rstd=None, eps: float = 1e-6, stream=None):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, of x bf16 or f32 [rows][k].

    residual (bf16 or f32 [rows][k]) may be absent.  Outputs, as wanted: residual_out (s, in
    residual's type; may be residual), y (bf16 or f32; may be x), q e4m3 with sfa (y as 1x128; k a
    multiple of 128), rstd f32 [rows] (for the backward pass)."""
    if _quick and _done(_quick.rms_norm(x, weight, residual, residual_out, y, q, sfa, rstd, eps, _number(stream)),
                        "fp8bs_rms_norm"):
        return
    index = _start(x, "x")
    xp, rows, k = _matrix(x, "x", _FLOAT, index)
    shape = x.shape
    wp = _like(weight, "weight", _FLOAT, (k,), index)
    rp = None if residual is None else _like(residual, "residual", _FLOAT, shape, index)
    op = None if residual_out is None else _like(residual_out, "residual_out", _FLOAT, shape, index)
    rt = residual if residual is not None else residual_out
    if rp is not None and op is not None and residual.dtype is not residual_out.dtype:
        raise TypeError("residual and residual_out must have the same dtype")
    yp = None if y is None else _like(y, "y", _FLOAT, shape, index)
    qp, sp = _codes(q, sfa, ("q", "sfa"), 1, rows, k, shape, index)
    tp = None if rstd is None else _like(rstd, "rstd", _F32, (rows,), index)
    if yp is None and qp is None and op is None and rows:
        raise ValueError("no output given: residual_out, y or q")
    _call("fp8bs_rms_norm", index, stream, xp, _CODE[x.dtype], rp, op,
          DTYPE_BF16 if rt is None else _CODE[rt.dtype], wp, _CODE[weight.dtype], yp,
          DTYPE_BF16 if y is None else _CODE[y.dtype], qp, sp, tp, rows, k, eps)


def rms_norm_1x128(x, weight, residual=None, eps: float = 1e-6, stream=None):
    """(q, sfa, s, rstd) of ``fp8bs_rms_norm``, new tensors; s is x where there is no residual."""
    index = _start(x, "x")
    _, rows, k = _matrix(x, "x", _FLOAT, index)
    q = _new((rows, k), _u8, index, stream)
    sfa = _new((k // 128, _ld(rows)), _f32, index, stream)
    rstd = _new((rows,), _f32, index, stream)
    s = None if residual is None else _new((rows, k), residual.dtype, index, stream)
    fp8bs_rms_norm(x, weight, residual, s, None, q, sfa, rstd, eps, stream)
    return q, sfa, x if s is None else s, rstd


@functools.lru_cache(256)
def rms_norm_backward_workspace_size(rows: int, k: int) -> int:
    _within("rms_norm_backward_workspace_size", k)
    return _size("fp8bs_rms_norm_backward_workspace_size", rows, k)


def fp8bs_rms_norm_backward(s, rstd, weight, dy, dx, dresidual=None, dweight=None,
                            accumulate: bool = False, workspace=None, stream=None):
    """Gradients of the norm: s bf16 or f32 [rows][k] (residual_out, or x without a residual) and
    rstd as the forward call gave it, dy bf16 or f32 -> dx in s's type (of x and of residual) and
    dweight f32 [k] (accumulate: added to what it holds), which may be None.  dresidual: the
    gradient of residual_out, in s's type; dx may be dresidual, s or dy.  workspace: uint8 tensor
    of rms_norm_backward_workspace_size() bytes, or None to allocate one."""
    if _quick and _done(_quick.rms_norm_backward(s, rstd, weight, dy, dx, dresidual, dweight, accumulate, workspace,
                                                 _number(stream)), "fp8bs_rms_norm_backward"):
        return
    index = _start(s, "s")
    sp, rows, k = _matrix(s, "s", _FLOAT, index)
    shape = s.shape
    tp = _like(rstd, "rstd", _F32, (rows,), index)
    wp = _like(weight, "weight", _FLOAT, (k,), index)
    gp = _like(dy, "dy", _FLOAT, shape, index)
    xp = _like(dx, "dx", (s.dtype,), shape, index)
    rp = None if dresidual is None else _like(dresidual, "dresidual", (s.dtype,), shape, index)
    dwp = None if dweight is None else _like(dweight, "dweight", _F32, (k,), index)
    p, n, _keep = None, 0, None
    if dwp is not None:
        p, n, _keep = _space(workspace, lambda: rms_norm_backward_workspace_size(rows, k), index,
                             stream)
    _call("fp8bs_rms_norm_backward", index, stream, sp, _CODE[s.dtype], tp, wp,
          _CODE[weight.dtype], gp, _CODE[dy.dtype], rp, xp, dwp, 1 if accumulate else 0, rows, k, p, n)


# ---- dispatch and combine ----------------------------------------------------------

def moe_capacity(tokens: int, topk: int, num_groups: int) -> int:
    """Rows of the contiguous layout that hold any choices."""
    _within("moe_capacity", topk, num_groups)
    return _size("fp8bs_moe_capacity", tokens, topk, num_groups)


@functools.lru_cache(256)
def moe_dispatch_workspace_size(layout: int, tokens: int, topk: int, num_groups: int,
                                m: int) -> int:
    """Workspace bytes of ``fp8bs_moe_dispatch`` (layout: LAYOUT_CONTIGUOUS or LAYOUT_MASKED; m:
    rows, of a slot if masked)."""
    _within("moe_dispatch_workspace_size", layout, topk, num_groups)
    return _size("fp8bs_moe_dispatch_workspace_size", layout, tokens, topk, num_groups, m)


def fp8bs_moe_dispatch(ids, x, a, group_data, positions, counts, sfx=None, sfa=None,
                       workspace=None, stream=None):
    """Tokens' rows to their experts: ids int32 or int64 [tokens][topk] (experts elsewhere: any
    number outside 0 .. g-1), x [tokens][k] e4m3 with sfx, bf16 or f32.

    a in x's type: [m][k] (contiguous layout; m at least moe_capacity()) with group_data the
    grouped_layout int32 [m], or [g][m][k] (masked) with group_data the masked_m int32 [g]; sfa its
    scales if e4m3.  positions int32 [tokens][topk]: each choice's row, -1 for none; counts int32
    [g]: choices of each expert.  workspace: uint8 tensor of moe_dispatch_workspace_size() bytes,
    or None to allocate one if it is needed."""
    if _quick and _done(_quick.moe_dispatch(ids, x, a, group_data, positions, counts, sfx, sfa, workspace,
                                            _number(stream)), "fp8bs_moe_dispatch"):
        return
    index = _start(ids, "ids")
    ip = _ptr(ids, "ids", _IDS, 2, index)
    tokens, topk = ids.shape
    xp, rows, k = _matrix(x, "x", _ROWS, index)
    if rows != tokens:
        raise ValueError("ids must have one row per row of x")
    cp = _ptr(counts, "counts", _INT32, 1, index)
    g = counts.shape[0]
    kind = _CODE[x.dtype]
    masked = isinstance(a, _Tensor) and a.ndim == 3
    ap = _ptr(a, "a", _FP8 if kind == DTYPE_E4M3 else (x.dtype,), 3 if masked else 2, index)
    m = a.shape[-2]
    _within("a", g, m, topk)
    if a.shape[-1] != k or (masked and a.shape[0] != g):
        raise ValueError("shape mismatch between x, a and counts")
    gp = _like(group_data, "group_data", _INT32, (g,) if masked else (m,), index)
    pp = _like(positions, "positions", _INT32, ids.shape, index)
    sxp = sap = None
    if kind == DTYPE_E4M3:
        sxp = _scales(sfx, "sfx", (k // 128) * _ld(tokens), index)
        sap = _scales(sfa, "sfa", (g if masked else 1) * (k // 128) * _ld(m), index)
    elif sfx is not None or sfa is not None:
        raise ValueError("sfx and sfa belong to e4m3 rows")
    layout = LAYOUT_MASKED if masked else LAYOUT_CONTIGUOUS
    wp, wb, _keep = _space(workspace, lambda: moe_dispatch_workspace_size(layout, tokens, topk, g,
                                                                          m), index, stream)
    _call("fp8bs_moe_dispatch", index, stream, layout, ip, ids.element_size(), xp, kind, sxp, ap,
          sap, gp, pp, cp, tokens, topk, g, m, k, wp, wb)


Dispatched = namedtuple("Dispatched", "a sfa group_data positions counts")


def moe_dispatch(ids, x, num_groups: int, sfx=None, max_m=None, stream=None):
    """``fp8bs_moe_dispatch`` into new tensors (a Dispatched tuple): the contiguous layout, or
    slots of max_m rows.  Rows that hold no token are not written."""
    index = _start(ids, "ids")
    _, tokens, k = _matrix(x, "x", _ROWS, index)
    if ids.ndim != 2:
        raise ValueError("ids must be [tokens][topk]")
    _within("ids", ids.shape[1], int(num_groups))
    g = int(num_groups)
    if g < 1:
        raise ValueError("num_groups must be at least 1")
    i32 = _INT32[0]
    if max_m is None:
        m = moe_capacity(tokens, ids.shape[1], g)
        lead, data = (m,), _new((m,), i32, index, stream)
    else:
        m = int(max_m)
        lead, data = (g, m), _new((g,), i32, index, stream)
    a = _new((*lead, k), x.dtype, index, stream)
    sfa = None
    if sfx is not None:
        sfa = _new((*lead[:-1], k // 128, _ld(m)), _f32, index, stream)
    out = Dispatched(a, sfa, data, _new(ids.shape, i32, index, stream),
                     _new((g,), i32, index, stream))
    fp8bs_moe_dispatch(ids, x, a, data, out.positions, out.counts, sfx, sfa, None, stream)
    return out


def _assigned(positions, weights, tokens, index):
    """(addresses of positions and weights, topk)"""
    pp = _ptr(positions, "positions", _INT32, 2, index)
    if positions.shape[0] != tokens:
        raise ValueError("positions must have one row per token")
    _within("positions", positions.shape[1])
    wp = None if weights is None else _like(weights, "weights", _F32, positions.shape, index)
    return pp, wp, positions.shape[1]


def fp8bs_moe_combine(d, positions, y, weights=None, stream=None):
    """y[t] = sum over j of weights[t][j] * d[positions[t][j]]: d bf16 [m][k] or [g][m][k],
    positions as dispatch gives them, weights f32 [tokens][topk] or None (ones: the gradient of
    dispatch), y bf16 or f32 [tokens][k]."""
    if _quick and _done(_quick.moe_combine(d, positions, y, weights, _number(stream)), "fp8bs_moe_combine"):
        return
    index = _start(d, "d")
    dp = _ptr(d, "d", (_bf16,), 3 if d.ndim == 3 else 2, index)
    yp, tokens, k = _matrix(y, "y", _FLOAT, index)
    if d.shape[-1] != k:
        raise ValueError("d and y must have the same number of columns")
    pp, wp, topk = _assigned(positions, weights, tokens, index)
    rows = d.shape[0] * d.shape[1] if d.ndim == 3 else d.shape[0]
    _call("fp8bs_moe_combine", index, stream, dp, pp, wp, yp, _CODE[y.dtype], rows, tokens, topk, k)


def fp8bs_moe_combine_backward(dy, positions, d=None, weights=None, dd=None, q=None, sfa=None,
                               dweights=None, stream=None):
    """Gradients of fp8bs_moe_combine: dy bf16 or f32 [tokens][k] -> the gradient of d as bf16
    (dd) or e4m3 (q, sfa), or both, at the rows that positions name, and dweights f32
    [tokens][topk] (needs d).  dd, q and d have the shape [m][k] or [g][m][k]."""
    if _quick and _done(_quick.moe_combine_backward(dy, positions, d, weights, dd, q, sfa, dweights, _number(stream)),
                        "fp8bs_moe_combine_backward"):
        return
    index = _start(dy, "dy")
    gp, tokens, k = _matrix(dy, "dy", _FLOAT, index)
    pp, wp, topk = _assigned(positions, weights, tokens, index)
    if dweights is not None and d is None:
        raise ValueError("dweights needs d")
    like = next((t for t in (dd, q, d) if t is not None), None)
    if like is None or (dd is None and q is None and dweights is None):
        raise ValueError("no output given: dd, q or dweights")
    shape = like.shape
    if len(shape) not in (2, 3) or shape[-1] != k:
        raise ValueError(f"dd, q and d must be [m][{k}] or [g][m][{k}], got {tuple(shape)}")
    slots, m = shape[0] if len(shape) == 3 else 1, shape[-2]
    _within("d", slots, m)
    dp = None if d is None else _like(d, "d", (_bf16,), shape, index)
    ddp = None if dd is None else _like(dd, "dd", (_bf16,), shape, index)
    qp, sp = _codes(q, sfa, ("q", "sfa"), slots, m, k, shape, index)
    dwp = None if dweights is None else _like(dweights, "dweights", _F32, positions.shape, index)
    _call("fp8bs_moe_combine_backward", index, stream, gp, _CODE[dy.dtype], dp, pp, wp, ddp, qp, sp,
          dwp, slots, m, tokens, topk, k)


# ---- gated activation ----------------------------------------------------------------

def _gated_columns(two_f):
    if two_f % 2:
        raise ValueError("g must hold 2f columns")
    return two_f // 2


def fp8bs_gated_quantize(g, hq, sfh, gq=None, sfg=None, grouped_layout=None, masked_m=None,
                         activation: str = "silu", stream=None):
    """h = act(gate) * up as e4m3 (hq, sfh: 1x128), g bf16 [m][2f] or with masked_m [slots][m][2f]
    (gate columns, then up columns); gq, sfg: g itself as e4m3, kept for the backward pass.  Rows
    that grouped_layout (int32 [m], -1) or masked_m (int32 [slots]) leaves out are not written."""
    if _quick and _done(_quick.gated_quantize(g, hq, sfh, gq, sfg, grouped_layout, masked_m,
                                              _mx.ACTIVATIONS.get(activation, -1), _number(stream)),
                        "fp8bs_gated_quantize"):
        return
    if grouped_layout is not None and masked_m is not None:
        raise ValueError("grouped_layout and masked_m exclude each other")
    index = _start(g, "g")
    masked = masked_m is not None
    gp = _ptr(g, "g", (_bf16,), 3 if masked else 2, index)
    slots, m = g.shape[0] if masked else 1, g.shape[-2]
    _within("g", slots, m)
    f = _gated_columns(g.shape[-1])
    if f > 1 << 23:
        raise FP8BSError(1, "g: at most 2^24 columns")
    act = _activation(activation)
    hp, hs = _codes(hq, sfh, ("hq", "sfh"), slots, m, f, (*g.shape[:-1], f), index)
    if hp is None:
        raise ValueError("hq is missing")
    kp, ks = _codes(gq, sfg, ("gq", "sfg"), slots, m, 2 * f, g.shape, index)
    layout, data = LAYOUT_DENSE, None
    if masked:
        layout, data = LAYOUT_MASKED, _like(masked_m, "masked_m", _INT32, (slots,), index)
    elif grouped_layout is not None:
        layout = LAYOUT_CONTIGUOUS
        data = _like(grouped_layout, "grouped_layout", _INT32, (m,), index)
    _call("fp8bs_gated_quantize", index, stream, layout, gp, hp, hs, kp, ks, data, m, f, slots, act)


def fp8bs_gated_quantize_backward(g, dh, sfg=None, d=None, dq=None, sfd=None, dqt=None, sfdt=None,
                                  hqt=None, sfht=None, grouped_layout=None,
                                  activation: str = "silu", stream=None):
    """Gradients of the gated activation at the checkpoint g e4m3 [m][2f] with sfg (or at g bf16),
    from dh bf16 [m][f].  Outputs, as wanted: d (bf16 [m][2f]), dq, sfd (e4m3, 1x128), dqt, sfdt
    (e4m3, 128x1: an operand of the weight gradient) and hqt, sfht (the activation h, 128x1)."""
    if _quick and _done(_quick.gated_quantize_backward(g, dh, sfg, d, dq, sfd, dqt, sfdt, hqt, sfht, grouped_layout,
                                                       _mx.ACTIVATIONS.get(activation, -1), _number(stream)),
                        "fp8bs_gated_quantize_backward"):
        return
    index = _start(g, "g")
    gp, m, two_f = _matrix(g, "g", _KEPT, index)
    f = _gated_columns(two_f)
    kind = _CODE[g.dtype]
    act = _activation(activation)
    sp = None
    if kind == DTYPE_E4M3:
        sp = _scales(sfg, "sfg", (two_f // 128) * _ld(m), index)
    elif sfg is not None:
        raise ValueError("sfg belongs to an e4m3 g")
    dhp = _like(dh, "dh", (_bf16,), (m, f), index)
    dp = None if d is None else _like(d, "d", (_bf16,), g.shape, index)
    qp, qs = _codes(dq, sfd, ("dq", "sfd"), 1, m, two_f, g.shape, index)
    tp, ts = _columns(dqt, sfdt, ("dqt", "sfdt"), m, two_f, index)
    hp, hs = _columns(hqt, sfht, ("hqt", "sfht"), m, f, index)
    if dp is None and qp is None and tp is None and hp is None and m:
        raise ValueError("no output given: d, dq, dqt or hqt")
    lp = None if grouped_layout is None else _like(grouped_layout, "grouped_layout", _INT32, (m,), index)
    _call("fp8bs_gated_quantize_backward", index, stream, gp, kind, sp, dhp, dp, qp, qs, tp, ts, hp,
          hs, lp, m, f, act)


# ---- quantiser along tokens ------------------------------------------------------------

def fp8bs_quantize_128x1(x, q, sf, sfx=None, grouped_layout=None, stream=None):
    """x [rows][n] f32, bf16 or e4m3 with sfx (1x128) -> q e4m3 [R][n], R = rows rounded up to a
    multiple of 128, and sf f32 [R/128][n]: an operand of fp8bs_k_grouped_tn_contiguous.  Rows
    that grouped_layout (int32 [rows], -1) leaves out are zeros."""
    if _quick and _done(_quick.quantize_128x1(x, q, sf, sfx, grouped_layout, _number(stream)), "fp8bs_quantize_128x1"):
        return
    index = _start(x, "x")
    xp, rows, n = _matrix(x, "x", _ROWS, index)
    kind = _CODE[x.dtype]
    sxp = None
    if kind == DTYPE_E4M3:
        sxp = _scales(sfx, "sfx", (n // 128) * _ld(rows), index)
    elif sfx is not None:
        raise ValueError("sfx belongs to an e4m3 x")
    qp, sp = _columns(q, sf, ("q", "sf"), rows, n, index)
    if qp is None:
        raise ValueError("q is missing")
    lp = None if grouped_layout is None else _like(grouped_layout, "grouped_layout", _INT32, (rows,), index)
    _call("fp8bs_quantize_128x1", index, stream, xp, kind, sxp, qp, sp, lp, rows, n)


def quantize_128x1(x, sfx=None, grouped_layout=None, stream=None):
    """(q, sf) of ``fp8bs_quantize_128x1``, new tensors."""
    index = _start(x, "x")
    _, rows, n = _matrix(x, "x", _ROWS, index)
    padded = (rows + 127) // 128 * 128
    q = _new((padded, n), _u8, index, stream)
    sf = _new((padded // 128, _ld(n)), _f32, index, stream)
    fp8bs_quantize_128x1(x, q, sf, sfx, grouped_layout, stream)
    return q, sf
