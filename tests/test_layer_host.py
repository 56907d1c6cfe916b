"""Host-side checks of the operators between the FP8 products (no GPU needed): sizes, pointers and
codes are refused before anything is launched, empty calls do nothing, sizes of workspaces, and
what the binding refuses."""
import ctypes

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs
import _layer_ref as ref

OK, SHAPE, POINTER, UNSUPPORTED = 0, 1, 2, 3
F32, BF16, E4M3 = 0, 1, 2
DENSE, CONTIGUOUS, MASKED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    return fp8bs.layer._load()


@pytest.fixture(scope="module")
def p():
    """a 16-byte aligned address; every call below fails before using it"""
    buf = ctypes.create_string_buffer(256)
    p.keep = buf
    return (ctypes.addressof(buf) + 15) // 16 * 16


def test_norm_refusals(lib, p):
    def norm(rows=4, k=128, x=p, xt=BF16, res=p, out=p, rt=BF16, w=p, wt=BF16, y=p, yt=BF16, q=p,
             sfa=p, rstd=p, eps=1e-6):
        return lib.fp8bs_rms_norm(x, xt, res, out, rt, w, wt, y, yt, q, sfa, rstd, rows, k, eps, None)

    for k in (0, -8, 4, 12, 100, 32776, 1 << 20):
        assert norm(k=k) == SHAPE
    assert norm(k=136) == SHAPE and norm(rows=-1) == SHAPE and norm(rows=0x7fffffff) == SHAPE
    for eps in (0.0, -1e-6, float("nan"), float("inf"), 1e-50):
        assert norm(eps=eps) == SHAPE
    for code in ("xt", "rt", "wt", "yt"):
        assert norm(**{code: 2}) == UNSUPPORTED and norm(**{code: -1}) == UNSUPPORTED
    assert norm(x=None) == POINTER and norm(w=None) == POINTER and norm(sfa=None) == POINTER
    for name in ("x", "res", "out", "w", "y", "q", "sfa"):
        assert norm(**{name: p + 8}) == POINTER, name
    assert norm(rstd=p + 2) == POINTER
    assert norm(out=None, y=None, q=None) == POINTER
    assert norm(rows=0, x=None, w=None, out=None, y=None, q=None) == OK


def test_norm_backward_refusals(lib, p):
    big = 1 << 40

    def back(rows=400, k=128, s=p, st=BF16, rstd=p, w=p, wt=BF16, dy=p, dt=BF16, dres=p, dx=p, dw=p,
             ws=p, n=big):
        return lib.fp8bs_rms_norm_backward(s, st, rstd, w, wt, dy, dt, dres, dx, dw, 0, rows, k, ws,
                                           n, None)

    for k in (0, 4, 100, 32776):
        assert back(k=k) == SHAPE
    assert back(rows=-1) == SHAPE
    assert back(st=2) == UNSUPPORTED and back(wt=3) == UNSUPPORTED and back(dt=-1) == UNSUPPORTED
    for name in ("s", "w", "dy", "dx", "rstd", "ws"):
        assert back(**{name: None}) == POINTER, name
    for name in ("s", "w", "dy", "dx", "dres", "dw", "ws"):
        assert back(**{name: p + 4}) == POINTER, name
    need = lib.fp8bs_rms_norm_backward_workspace_size(400, 128)
    assert need > 0 and back(n=need - 1) == UNSUPPORTED
    assert back(rows=0, s=None, rstd=None, w=None, dy=None, dx=None, dw=None, ws=None, n=0) == OK
    size = lib.fp8bs_rms_norm_backward_workspace_size
    assert size(-1, 128) == -SHAPE and size(4, 100) == -SHAPE and size(0, 128) == 0
    assert size(384, 7168) == 0 and size(385, 7168) == 256 * 7168 * 4    # few rows need none
    # no more than 512 parts, whatever the rows
    assert size(1 << 30, 7168) == size(1 << 20, 7168) == 512 * 7168 * 4


def test_dispatch_refusals(lib, p):
    big = 1 << 40

    def dispatch(layout=CONTIGUOUS, ids=p, w=4, x=p, xt=E4M3, sfx=p, a=p, sfa=p, data=p, pos=p,
                 counts=p, tokens=8, topk=2, g=4, m=512, k=128, ws=p, n=big):
        return lib.fp8bs_moe_dispatch(layout, ids, w, x, xt, sfx, a, sfa, data, pos, counts, tokens,
                                      topk, g, m, k, ws, n, None)

    assert dispatch(layout=DENSE) == UNSUPPORTED and dispatch(layout=3) == UNSUPPORTED
    assert dispatch(w=2) == UNSUPPORTED and dispatch(xt=3) == UNSUPPORTED
    for k in (0, 64, 130, (1 << 24) + 128):
        assert dispatch(k=k) == SHAPE
    assert dispatch(k=12, xt=BF16) == SHAPE
    assert dispatch(tokens=-1) == SHAPE and dispatch(topk=0) == SHAPE and dispatch(topk=65) == SHAPE
    assert dispatch(g=0) == SHAPE and dispatch(g=1025) == SHAPE
    assert dispatch(tokens=(1 << 30) // 2 + 1, m=0x7fffff00 // 128 * 128) == SHAPE
    # 16 choices over four experts can need 16 + 4 x 127 rows: 384, or 512 where they are uneven
    assert lib.fp8bs_moe_capacity(8, 2, 4) == 512
    assert dispatch(m=384) == SHAPE and dispatch(m=513) == SHAPE and dispatch(m=-128) == SHAPE
    assert dispatch(layout=MASKED, m=-1) == SHAPE
    assert dispatch(layout=MASKED, m=0x7fffff00, g=2) == SHAPE
    for name in ("ids", "x", "sfx", "a", "sfa", "data", "pos", "counts"):
        assert dispatch(**{name: None}) == POINTER, name
        assert dispatch(**{name: p + 2}) == POINTER, name
    assert dispatch(w=8, ids=p + 4) == POINTER
    many = dict(tokens=4096, topk=8, m=64 * 1024)
    need = lib.fp8bs_moe_dispatch_workspace_size(CONTIGUOUS, 4096, 8, 4, 64 * 1024)
    assert need > 0 and dispatch(**many, n=need - 1) == UNSUPPORTED
    assert dispatch(**many, ws=None) == POINTER and dispatch(**many, ws=p + 8) == POINTER
    size = lib.fp8bs_moe_dispatch_workspace_size
    assert size(DENSE, 4, 2, 4, 512) == -UNSUPPORTED and size(MASKED, 4, 0, 4, 512) == -SHAPE
    assert size(MASKED, 4, 2, 4, -1) == -SHAPE
    # refused sizes do not wrap around
    assert size(MASKED, 1 << 24, 64, 1024, 0x7fffff00) > 1 << 40


def test_capacity_holds_the_worst_choices(lib):
    for tokens, topk, g in [(0, 1, 8), (1, 1, 8), (1, 8, 8), (16, 2, 1), (7, 3, 5), (300, 8, 256)]:
        n = tokens * topk
        cap = fp8bs.moe_capacity(tokens, topk, g)
        # as many experts as possible with one choice more than a multiple of 128
        worst, left, experts = 0, n, 0
        while left and experts < g:
            take = 1 if experts < g - 1 else left
            worst += (take + 127) // 128 * 128
            left -= take
            experts += 1
        assert cap % 128 == 0 and cap >= worst
        rng = np.random.default_rng(n)
        for _ in range(20):
            ids = rng.integers(0, g, (tokens, topk))
            counts = np.bincount(ids.reshape(-1), minlength=g)
            assert ((counts + 127) // 128 * 128).sum() <= cap
    size = lib.fp8bs_moe_capacity
    assert size(-1, 2, 4) == -SHAPE and size(1 << 30, 2, 4) == -SHAPE and size(1, 65, 4) == -SHAPE
    assert size(4, 2, 0) == -SHAPE


def test_combine_refusals(lib, p):
    def combine(d=p, pos=p, w=p, y=p, yt=BF16, rows=64, tokens=4, topk=2, k=128):
        return lib.fp8bs_moe_combine(d, pos, w, y, yt, rows, tokens, topk, k, None)

    def back(dy=p, dt=BF16, d=p, pos=p, w=p, dd=p, q=p, sfa=p, dw=p, slots=2, m=32, tokens=4, topk=2,
             k=128):
        return lib.fp8bs_moe_combine_backward(dy, dt, d, pos, w, dd, q, sfa, dw, slots, m, tokens,
                                              topk, k, None)

    for call in (combine, back):
        for k in (0, 4, 100, 1 << 25):
            assert call(k=k) == SHAPE
        assert call(tokens=-1) == SHAPE and call(topk=0) == SHAPE and call(topk=65) == SHAPE
        assert call(pos=None) == POINTER and call(pos=p + 2) == POINTER and call(w=p + 2) == POINTER
        assert call(d=None) == POINTER and call(d=p + 8) == POINTER
    assert combine(rows=-1) == SHAPE and combine(rows=1 << 31) == SHAPE
    assert combine(yt=E4M3) == UNSUPPORTED and back(dt=E4M3) == UNSUPPORTED
    assert combine(y=None) == POINTER and combine(y=p + 8) == POINTER
    assert combine(tokens=0, d=None, pos=None, y=None) == OK
    assert back(k=136) == SHAPE and back(slots=0) == SHAPE and back(m=-1) == SHAPE
    assert back(slots=3, m=0x7fffff00) == SHAPE
    for name in ("dy", "dd", "q", "sfa", "dw"):
        assert back(**{name: p + 2}) == POINTER, name
    assert back(dy=None) == POINTER and back(sfa=None) == POINTER
    assert back(dd=None, q=None, dw=None) == POINTER
    assert back(tokens=0, dy=None, pos=None) == OK


def test_gated_refusals(lib, p):
    def gated(layout=DENSE, g=p, hq=p, sfh=p, gq=p, sfg=p, data=p, m=4, f=128, groups=2, act=0):
        return lib.fp8bs_gated_quantize(layout, g, hq, sfh, gq, sfg, data, m, f, groups, act, None)

    def back(g=p, gt=E4M3, sfg=p, dh=p, d=p, dq=p, sfd=p, dqt=p, sfdt=p, hqt=p, sfht=p, lay=None, m=4,
             f=128, act=0):
        return lib.fp8bs_gated_quantize_backward(g, gt, sfg, dh, d, dq, sfd, dqt, sfdt, hqt, sfht,
                                                 lay, m, f, act, None)

    for call in (gated, back):
        for f in (0, 64, 130, (1 << 20) + 128):
            assert call(f=f) == SHAPE
        assert call(m=-1) == SHAPE and call(m=0x7fffffff) == SHAPE
        assert call(act=2) == UNSUPPORTED and call(act=-1) == UNSUPPORTED
        assert call(g=None) == POINTER and call(g=p + 8) == POINTER and call(sfg=None) == POINTER
        assert call(m=0x7fffff00, f=1 << 20) == UNSUPPORTED
    assert gated(layout=3) == UNSUPPORTED and gated(layout=MASKED, groups=0) == SHAPE
    assert gated(layout=CONTIGUOUS, m=100) == SHAPE and back(lay=p, m=100) == SHAPE
    for layout in (CONTIGUOUS, MASKED):
        assert gated(layout=layout, m=128, data=None) == POINTER
    for name in ("hq", "sfh"):
        assert gated(**{name: None}) == POINTER
    assert gated(m=0, g=None, hq=None, sfh=None, gq=None, sfg=None) == OK
    assert back(gt=F32) == UNSUPPORTED and back(dh=None) == POINTER
    for name in ("sfd", "sfdt", "sfht"):
        assert back(**{name: None}) == POINTER, name
    for name in ("d", "dq", "sfd", "dqt", "sfdt", "hqt", "sfht", "dh"):
        assert back(**{name: p + 8}) == POINTER, name
    assert back(lay=p + 2, m=128) == POINTER
    assert back(d=None, dq=None, dqt=None, hqt=None) == POINTER
    assert back(m=0, g=None, dh=None, d=None, dq=None, dqt=None, hqt=None) == OK


def test_columns_refusals(lib, p):
    def columns(x=p, xt=BF16, sfx=p, q=p, sf=p, lay=None, rows=4, n=128):
        return lib.fp8bs_quantize_128x1(x, xt, sfx, q, sf, lay, rows, n, None)

    for n in (0, 8, 24, (1 << 20) + 16):
        assert columns(n=n) == SHAPE
    assert columns(xt=E4M3, n=144) == SHAPE and columns(rows=-1) == SHAPE
    assert columns(rows=100, lay=p) == SHAPE and columns(xt=3) == UNSUPPORTED
    assert columns(rows=0x7fffff00, n=1 << 20) == UNSUPPORTED
    for name in ("x", "q", "sf"):
        assert columns(**{name: None}) == POINTER and columns(**{name: p + 8}) == POINTER
    assert columns(xt=E4M3, sfx=None) == POINTER and columns(lay=p + 2, rows=128) == POINTER
    assert columns(rows=0, x=None, q=None, sf=None) == OK


def test_the_binding_refuses_host_tensors_and_other_types():
    x, w = torch.zeros(4, 128), torch.zeros(128)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_rms_norm(x, w, y=x)
    with pytest.raises(TypeError):
        fp8bs.fp8bs_rms_norm([1.0], w, y=x)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_rms_norm_backward(x, w, w, x, x)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_moe_dispatch(ids, x, x, ids, ids, ids)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_moe_combine(x, ids, x)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_moe_combine_backward(x, ids, dd=x)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_gated_quantize(x, x, x)
    with pytest.raises(ValueError, match="exclude"):
        fp8bs.fp8bs_gated_quantize(x, x, x, grouped_layout=ids, masked_m=ids)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_gated_quantize_backward(x, x)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_quantize_128x1(x, x, x)


def test_sizes_that_an_int_does_not_hold_are_refused():
    """they would wrap to small ones: 2^32 + 1 rows to one row (the pages of the tensors here are
    never touched)"""
    m = fp8bs.layer
    m._load()
    many = (1 << 32) + 1
    tall = torch.empty(many, 1, dtype=torch.uint8)
    with pytest.raises(fp8bs.FP8BSError, match="2.31"):
        m._matrix(tall, "x", m._ROWS, tall.get_device())
    for t in (torch.empty(8, 16, dtype=torch.uint8), torch.empty(0, 16, dtype=torch.uint8)):
        assert m._matrix(t, "x", m._ROWS, t.get_device())[1:] == tuple(t.shape)
    for call in (lambda: m.moe_capacity(1, many, 8), lambda: m.moe_capacity(1, 1, many),
                 lambda: m.moe_dispatch_workspace_size(CONTIGUOUS, 1, many, 8, 128),
                 lambda: m.rms_norm_backward_workspace_size(8, (1 << 32) + 8),
                 lambda: m._within("g", 1, many)):
        with pytest.raises(fp8bs.FP8BSError):
            call()


def test_the_compiled_module_takes_device_tensors_alone(monkeypatch):
    m = fp8bs.layer
    m._load()
    t = torch.zeros(4, 128)
    for name, count in (("rms_norm", 10), ("rms_norm_backward", 10), ("moe_dispatch", 10), ("moe_combine", 5),
                        ("moe_combine_backward", 9), ("gated_quantize", 9), ("gated_quantize_backward", 13),
                        ("quantize_128x1", 6)):
        call = getattr(m._quick, name)
        for operand in (t, None, 1, "x", torch.nn.Parameter(t), t.numpy()):
            assert call(*[operand] * count) == -1, (name, operand)
        assert call() == -1 and call(*[t] * (count + 1)) == -1
    with pytest.raises(TypeError):
        m._quick.use(1, 2)
    with pytest.raises(TypeError):
        m._quick.use(*["x"] * 11)
    with pytest.raises(ValueError, match="device"):
        fp8bs.fp8bs_rms_norm(t, t[0], y=t)
    monkeypatch.setattr(m, "_MODULE_PATH", "/nowhere/fp8bs_layer_py.so")
    with pytest.raises(RuntimeError, match="build it"):
        m._load_module(m._lib)


def test_the_reference_quantiser():
    """the tests' own quantiser against torch's cast, and its half step"""
    rng = np.random.default_rng(1)
    v = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.uniform(-4, 2.6, 4000),
                        ref._MID, -ref._MID, ref.VALUES[np.isfinite(ref.VALUES)]]).astype(np.float32)
    v = np.clip(v, -448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.codes(v), want)
    x = rng.normal(size=(256, 256)).astype(np.float32)
    for axis in (0, -1):
        q, s = ref.quantise(x, axis)
        ref.check_quantised(q, s, x.astype(np.float64), np.zeros(x.shape), axis, axis)
        worse = q.copy()
        worse[3, 5] ^= 1
        with pytest.raises(AssertionError):
            ref.check_quantised(worse, s, x.astype(np.float64), np.zeros(x.shape), axis, axis)
