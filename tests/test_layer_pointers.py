"""Operands that dispatch reads although nothing is written: refused on the host where they are
missing (no GPU needed, each call fails before a launch)."""
import ctypes

import pytest

import moe_grouped_gemm_block_amd as fp8bs

POINTER = 2
BF16, E4M3 = 1, 2
MASKED = 2


@pytest.fixture(scope="module")
def lib():
    return fp8bs.layer._load()


@pytest.fixture(scope="module")
def p():
    """a 16-byte aligned address that no call below uses"""
    buf = ctypes.create_string_buffer(256)
    p.keep = buf
    return (ctypes.addressof(buf) + 15) // 16 * 16


# one launch, whose workgroups fetch a token's scales before they know its rows, and three
@pytest.mark.parametrize("tokens,topk", [(1, 1), (8, 2), (512, 8), (4096, 8)])
def test_scales_of_rows_into_slots_of_none(lib, p, tokens, topk):
    def dispatch(m, sfx, a=None, sfa=None, x=p, kind=E4M3):
        return lib.fp8bs_moe_dispatch(MASKED, p, 4, x, kind, sfx, a, sfa, p, p, p, tokens, topk, 4, m, 128,
                                      p, 1 << 40, None)

    assert dispatch(0, None) == POINTER
    assert dispatch(0, p + 8) == POINTER
    assert dispatch(0, p, x=None) == POINTER and dispatch(0, None, x=None, kind=BF16) == POINTER
    assert dispatch(16, None, p, p) == POINTER
    assert dispatch(16, p, None, p) == POINTER and dispatch(16, p, p, None) == POINTER
