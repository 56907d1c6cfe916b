"""Host-side checks of the MXFP4 calls (no GPU needed): sizes, pointers and codes are refused
before anything is launched, empty calls do nothing, and the binding refuses what it cannot
pass on."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_block_amd as fp8bs

OK, SHAPE, POINTER, UNSUPPORTED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return fp8bs.mxfp4._load()


@pytest.fixture(scope="module")
def p():
    """a 16-byte aligned address; every call below fails before using it"""
    buf = ctypes.create_string_buffer(256)
    p.keep = buf
    return (ctypes.addressof(buf) + 15) // 16 * 16


def test_quantiser_refusals(lib, p):
    for call in (lambda x, dt, q, s, g, r, k: lib.fp8bs_quantize_mxfp4(x, dt, q, s, g, r, k, None),
                 lambda x, dt, q, s, g, r, k: lib.fp8bs_dequantize_mxfp4(q, s, x, dt, g, r, k, None)):
        assert call(p, 1, p, p, 1, 4, 100) == SHAPE
        assert call(p, 1, p, p, 1, 4, 0) == SHAPE
        assert call(p, 1, p, p, 1, -1, 128) == SHAPE
        assert call(p, 1, p, p, 0, 4, 128) == SHAPE
        assert call(p, 1, p, p, 1 << 20, 1 << 20, 1 << 20) == SHAPE
        # tiles past the last column or row would have numbers past 32 bits
        assert call(p, 1, p, p, 1, 1, (1 << 31) - 128) == SHAPE
        assert call(p, 1, p, p, 1, 0, (1 << 24) + 128) == SHAPE
        assert call(p, 1, p, p, 1, 0x7fffffff, 128) == SHAPE
        assert call(p, 2, p, p, 1, 4, 128) == UNSUPPORTED
        assert call(None, 1, p, p, 1, 4, 128) == POINTER
        assert call(p, 1, p + 4, p, 1, 4, 128) == POINTER
        assert call(p, 1, p, p + 4, 1, 4, 128) == POINTER
        assert call(None, 1, None, None, 1, 0, 128) == OK


def test_product_refusals(lib, p):
    def dense(m, n, k, a=p, sa=p, b=p, sb=p, d=p):
        return lib.fp8bs_dense_nt_mxfp4(a, sa, b, sb, d, m, n, k, None)

    def contiguous(m, n, k, g, lay=p):
        return lib.fp8bs_grouped_contiguous_nt_mxfp4(p, p, p, p, p, lay, m, n, k, g, None)

    def masked(g, m, n, k, mm=p):
        return lib.fp8bs_grouped_masked_nt_mxfp4(p, p, p, p, p, mm, g, m, 0, n, k, None)

    assert dense(4, 8, 64) == SHAPE and dense(4, 8, 192) == SHAPE and dense(4, 0, 128) == SHAPE
    assert dense(-1, 8, 128) == SHAPE and dense(4, 8, 1 << 25) == SHAPE
    assert dense(0x7fffffff, 8, 128) == SHAPE and dense(1 << 29, 8, 1024) == SHAPE
    assert dense(4, 8, 128, a=None) == POINTER and dense(4, 8, 128, sa=p + 4) == POINTER
    assert dense(4, 8, 128, b=p + 8) == POINTER and dense(4, 8, 128, sb=None) == POINTER
    assert dense(4, 8, 128, d=p + 2) == POINTER
    assert contiguous(100, 8, 128, 2) == SHAPE and contiguous(128, 8, 128, 0) == SHAPE
    assert contiguous(128, 8, 128, 2, None) == POINTER
    assert contiguous(128, 8, 128, 2, p + 2) == POINTER
    assert masked(0, 4, 8, 128) == SHAPE and masked(2, 4, 8, 130) == SHAPE
    assert masked(2, 4, 8, 128, None) == POINTER
    assert dense(0, 8, 128, None, None, None, None, None) == OK
    assert contiguous(0, 8, 128, 2, None) == OK and masked(2, 0, 8, 128, None) == OK


def test_gated_refusals(lib, p):
    def gated(m, f, k, act=0, h=p):
        return lib.fp8bs_gated_dense_mxfp4(p, p, p, p, h, m, f, k, act, None)

    def quantised(m, f, k, act=0, hq=p, sfh=p):
        return lib.fp8bs_gated_dense_mxfp4_q(p, p, p, p, hq, sfh, m, f, k, act, None)

    assert gated(4, 0, 128) == SHAPE and gated(4, 48, 128) == SHAPE and gated(4, 32, 100) == SHAPE
    assert gated(4, 32, 128, 2) == UNSUPPORTED and gated(4, 32, 128, -1) == UNSUPPORTED
    assert gated(4, 32, 128, 0, None) == POINTER
    assert quantised(4, 32, 128) == SHAPE and quantised(4, 192, 128) == SHAPE
    assert quantised(4, 128, 128, 0, None) == POINTER
    assert quantised(4, 128, 128, 0, p, p + 4) == POINTER
    assert lib.fp8bs_gated_contiguous_mxfp4(p, p, p, p, p, None, 128, 32, 128, 2, 0, None) == POINTER
    assert lib.fp8bs_gated_contiguous_mxfp4(p, p, p, p, p, p, 130, 32, 128, 2, 0, None) == SHAPE
    assert lib.fp8bs_gated_masked_mxfp4(p, p, p, p, p, None, 2, 4, 0, 32, 128, 0, None) == POINTER
    assert gated(0, 32, 128) == OK


def test_backward_refusals(lib, p):
    size = fp8bs.gated_backward_workspace_size

    def back(m=4, f=32, k=128, dh=p, da=p, db=p, dt=1, acc=0, act=0, ws=p, n=1 << 40):
        return lib.fp8bs_gated_dense_mxfp4_backward(p, p, p, p, dh, da, db, dt, acc, m, f, k, act,
                                                    ws, n, None)

    assert back(f=33) == SHAPE and back(k=64) == SHAPE and back(m=-1) == SHAPE
    assert back(act=7) == UNSUPPORTED and back(dt=2) == UNSUPPORTED
    assert back(dt=1, acc=1) == UNSUPPORTED                 # bf16 cannot be added to
    assert back(dh=None) == POINTER and back(da=p + 2) == POINTER and back(db=p + 4) == POINTER
    assert back(ws=None) == POINTER and back(ws=p + 8) == POINTER
    assert back(n=size(0, 4, 32, 128) - 1) == UNSUPPORTED
    assert back(da=None, db=None) == OK and back(m=0, db=None) == OK
    both = size(fp8bs.LAYOUT_CONTIGUOUS, 256, 64, 128, 3)
    da = size(fp8bs.LAYOUT_CONTIGUOUS, 256, 64, 128, 3, want_db=False)
    db = size(fp8bs.LAYOUT_CONTIGUOUS, 256, 64, 128, 3, want_da=False)
    # dg | du in bf16, and for db the blocks by expert
    assert both == db > da >= 256 * 128 * 2
    assert size(fp8bs.LAYOUT_DENSE, 65, 64, 128) >= 128 * 128 * 2       # rows to a multiple of 64
    assert size(fp8bs.LAYOUT_DENSE, 4, 32, 128, want_da=False, want_db=False) == 0
    assert size(fp8bs.LAYOUT_DENSE, 0, 32, 128, want_db=False) >= 0
    for bad in ((fp8bs.LAYOUT_MASKED, 128, 32, 128), (fp8bs.LAYOUT_CONTIGUOUS, 100, 32, 128),
                (fp8bs.LAYOUT_DENSE, 4, 31, 128), (fp8bs.LAYOUT_DENSE, 4, 32, 127)):
        with pytest.raises(fp8bs.FP8BSError):
            size(*bad)


def test_layer_refusals(lib, p):
    size = fp8bs.feed_forward_workspace_size

    def layer(layout=0, x=p, dt=1, d=p, data=p, m=4, f=128, k=128, n=8, g=2, act=0, ws=p, nb=1 << 40):
        return lib.fp8bs_feed_forward_mxfp4(layout, x, dt, p, p, p, p, d, data, m, 0, f, k, n, g, act,
                                            ws, nb, None)

    assert layer(layout=3) == SHAPE and layer(f=64) == SHAPE and layer(k=64) == SHAPE
    assert layer(n=0) == SHAPE and layer(m=-1) == SHAPE and layer(layout=2, g=0) == SHAPE
    assert layer(layout=1, m=100) == SHAPE
    assert layer(dt=5) == UNSUPPORTED and layer(act=2) == UNSUPPORTED
    assert layer(x=None) == POINTER and layer(d=p + 2) == POINTER and layer(ws=None) == POINTER
    assert layer(layout=2, data=None) == POINTER and layer(layout=1, m=128, data=p + 1) == POINTER
    assert layer(nb=size(0, 4, 128, 128) - 1) == UNSUPPORTED
    assert layer(m=0, x=None, d=None, ws=None, nb=0) == OK
    assert size(fp8bs.LAYOUT_MASKED, 16, 256, 384, 5) >= 5 * 16 * (192 + 128)
    for bad in ((3, 4, 128, 128), (fp8bs.LAYOUT_DENSE, 4, 96, 128), (fp8bs.LAYOUT_MASKED, 4, 128, 128, 0)):
        with pytest.raises(fp8bs.FP8BSError):
            size(*bad)


def test_binding_refuses_host_tensors_and_unknown_activations():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fp8bs.quantize_mxfp4(x)
    with pytest.raises(ValueError):
        fp8bs.quantize_mxfp4(torch.zeros(128))
    a, sf = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_dense_nt_mxfp4(a, sf, a, sf, torch.zeros(4, 4, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        fp8bs.fp8bs_dense_nt_mxfp4(None, sf, a, sf, x)
    with pytest.raises(ValueError):
        fp8bs.mxfp4._activation("relu")


@pytest.mark.gpu
def test_binding_refuses_mismatched_tensors():
    def u8(*s):
        return torch.zeros(s, dtype=torch.uint8, device="cuda")

    def i32(*s):
        return torch.zeros(s, dtype=torch.int32, device="cuda")

    def bf(*s):
        return torch.zeros(s, dtype=torch.bfloat16, device="cuda")

    a, sa, b, sb = u8(4, 64), i32(1, 4), u8(8, 64), i32(1, 8)
    ok = (a, sa, b, sb)
    for args, kind in (((a, sa, u8(8, 128), i32(2, 8), bf(4, 8)), ValueError),   # other k
                       ((a, i32(1, 8), b, sb, bf(4, 8)), ValueError),            # exponents' size
                       ((*ok, bf(4, 7)), ValueError),                            # d's shape
                       ((*ok, bf(8, 8)[::2]), ValueError),                       # strides
                       ((*ok, torch.zeros(4, 8, device="cuda")), TypeError),     # d's type
                       ((a.int(), sa, b, sb, bf(4, 8)), TypeError),
                       ((*ok, torch.zeros(4, 8, dtype=torch.bfloat16)), ValueError)):
        with pytest.raises(kind):
            fp8bs.fp8bs_dense_nt_mxfp4(*args)
    with pytest.raises(fp8bs.FP8BSError) as e:
        fp8bs.fp8bs_dense_nt_mxfp4(u8(4, 32), i32(1, 4), u8(8, 32), i32(1, 8), bf(4, 8))
    assert e.value.status == SHAPE
    w, sw = u8(64, 64), i32(1, 64)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_dense_mxfp4(a, sa, w, sw, bf(4, 64))
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_dense_mxfp4(a, sa, w, sw, bf(4, 32), activation="relu")
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_dense_mxfp4_backward(a, sa, w, sw, bf(4, 32), bf(4, 128), bf(64, 128),
                                               accumulate=True)
    with pytest.raises(ValueError):
        fp8bs.fp8bs_gated_dense_mxfp4_backward(a, sa, w, sw, bf(4, 31), bf(4, 128), None)
    with pytest.raises(fp8bs.FP8BSError) as e:
        fp8bs.fp8bs_gated_dense_mxfp4_backward(a, sa, w, sw, bf(4, 32), bf(4, 128), None,
                                               workspace=u8(16))
    assert e.value.status == UNSUPPORTED
    with pytest.raises(ValueError):
        fp8bs.fp8bs_grouped_contiguous_nt_mxfp4(u8(128, 64), i32(1, 128), u8(2, 8, 64), i32(2, 1, 8),
                                                bf(128, 8), i32(127))
    with pytest.raises(ValueError):
        fp8bs.fp8bs_grouped_masked_nt_mxfp4(u8(2, 4, 64), i32(2, 1, 4), u8(3, 8, 64),
                                            i32(3, 1, 8), bf(2, 4, 8), i32(2))
    with pytest.raises(ValueError):
        fp8bs.feed_forward_mxfp4(bf(4, 128), w, sw, w, sw, grouped_layout=i32(4), masked_m=i32(1))
