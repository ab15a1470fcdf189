"""Refusals of the low-bit entry points (host checks, nothing is launched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._build_module().build()
    from mixture_experts_grouped_router_gb300 import _lib
    return _lib


def P(v=4096):
    return ctypes.c_void_p(v)


BIG = 1 << 30


def test_scale_bytes(L):
    f = L.moe_fp4_scale_bytes
    assert f(100, 256, L.FP4_MX, L.FP4_ROWS_GROUPED, 4) == (100 + 4 * 127 + 127) // 128 * 2 * 512
    assert f(100, 256, L.FP4_NV, L.FP4_ROWS_GROUPED, 4) == (100 + 4 * 127 + 127) // 128 * 4 * 512
    assert f(3 * 200, 96, L.FP4_NV, L.FP4_ROWS_EXPERTS, 3) == 3 * 2 * 2 * 512
    assert f(2 * 448, 96, L.FP4_MX, L.FP4_ROWS_SWIGLU, 2) == 2 * 4 * 1 * 512
    assert f(-1, 96, 0, 1, 2) == 0 and f(8, 96, 7, 1, 2) == 0 and f(8, 96, 0, 0, 2) == 0
    assert f(0, 96, 0, L.FP4_ROWS_EXPERTS, 2) == 0


def quantize(L, x=P(), ldx=64, src=10, idx=None, div=1, rows=10, cols=64, fmt=0, m=1, off=P(), E=2,
             q=P(), ldq=32, sf=P(), nb=BIG, ws=None, wsb=0):
    return L.LIB.moe_fp4_quantize(x, ldx, src, idx, div, rows, cols, fmt, m, off, E, None, q, ldq,
                                  sf, nb, ws, wsb, None, None)


def test_fp4_quantize(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    assert quantize(L, fmt=2) == bad and "fmt" in L.last_error()
    assert quantize(L, m=0) == bad and "row_map" in L.last_error()
    assert quantize(L, cols=48, ldx=48) == uns and "32" in L.last_error()
    assert quantize(L, rows=-1) == bad
    assert quantize(L, off=None) == bad and "group_offsets" in L.last_error()
    assert quantize(L, E=257) == uns
    assert quantize(L, m=3, E=3, off=None) == bad and "equal groups" in L.last_error()
    assert quantize(L, m=2, E=1, off=None) == uns and "SWIGLU" in L.last_error()
    assert quantize(L, ldx=32) == bad and quantize(L, ldq=16) == bad
    assert quantize(L, ldx=68) == uns and quantize(L, ldq=40) == uns
    assert quantize(L, src=9) == bad
    assert quantize(L, idx=P(), div=0) == bad and "index_div" in L.last_error()
    assert quantize(L, q=None) == bad and quantize(L, x=P(4100)) == uns
    assert quantize(L, ws=P(4100), wsb=BIG) == uns
    assert quantize(L, nb=512) == bad and "sf of 512" in L.last_error()
    assert quantize(L, rows=0, x=None, q=None, sf=None, off=None) == L.MOE_OK


def test_fp4_dequantize_weights_scales(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    d = L.LIB.moe_fp4_dequantize
    assert d(P(), 32, P(), BIG, 10, 64, 0, 1, P(), 2, None, P(), 48, None) == bad
    assert d(P(), 32, P(), 16, 10, 64, 0, 1, P(), 2, None, P(), 64, None) == bad
    assert d(P(), 32, P(), BIG, 10, 64, 0, 1, P(), 2, None, None, 64, None) == bad
    assert d(P(), 32, P(), BIG, 10, 64, 0, 1, P(), 2, None, P(4098), 64, None) == uns
    w = L.LIB.moe_fp4_quantize_weights
    assert w(P(), 2, 64, 64, 0, 1, None, P(), P(), BIG, None) == bad
    assert w(P(), 2, 48, 64, 0, 3, None, P(), P(), BIG, None) == uns
    assert w(P(), 2, 64, 0, 0, 3, None, P(), P(), BIG, None) == bad
    assert w(P(), 2, 64, 96, 0, 2, None, P(), P(), BIG, None) == uns
    assert w(P(), 2, 64, 64, 0, 3, None, P(), P(), 8, None) == bad
    a = L.LIB.moe_fp4_arrange_scales
    assert a(P(), 64, 64, 0, 1, 2, P(), BIG, None) == bad
    assert a(P(), 65, 64, 0, 3, 2, P(), BIG, None) == bad
    assert a(None, 64, 64, 0, 3, 2, P(), BIG, None) == bad
    assert a(P(), 64, 64, 0, 3, 2, P(), 8, None) == bad


def gmm(L, A=P(), lda=32, B=P(), ldb=32, sb=32 * 64, fmt=1, off=P(), E=2, cap=10, K=64, N=64, epi=0,
        C=P(), dt=0, ldc=64, Q2=None, ldq2=0, sf2=None, nb=0):
    return L.LIB.moe_gmm_fp4(A, lda, P(), None, B, ldb, sb, P(), None, fmt, off, E, cap, K, N, epi,
                             C, dt, ldc, Q2, ldq2, sf2, nb, None, None, None)


def test_gmm_fp4(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    assert gmm(L, K=0) == bad and gmm(L, E=0) == bad and gmm(L, E=300) == uns
    assert gmm(L, fmt=3) == bad and gmm(L, epi=2) == bad and gmm(L, dt=5) == bad
    assert gmm(L, K=48) == uns and gmm(L, N=60) == uns and gmm(L, lda=40) == uns
    assert gmm(L, lda=16) == bad and gmm(L, ldb=16) == bad and gmm(L, sb=64) == bad
    assert gmm(L, ldc=56) == bad and gmm(L, dt=1, ldc=66) == bad
    assert gmm(L, C=None) == bad and gmm(L, off=None) == bad
    assert gmm(L, A=P(4104)) == uns
    assert gmm(L, cap=1 << 23) == uns
    sw = dict(epi=1, C=None, Q2=P(), ldq2=16, sf2=P(), nb=BIG)
    assert gmm(L, **dict(sw, N=96, sb=32 * 96)) == uns
    assert gmm(L, **dict(sw, dt=1)) == bad
    assert gmm(L, **dict(sw, ldq2=8)) == bad and gmm(L, **dict(sw, Q2=None)) == bad
    assert gmm(L, **dict(sw, nb=512)) == bad and "sf2" in L.last_error()
    assert gmm(L, cap=0, A=None, C=None, ldc=64) == L.MOE_OK


def test_act8(L):
    bad, uns = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    q = L.LIB.moe_act8_quantize
    assert q(P(), 64, -1, 64, None, 0, P(), 64, P(), 2, None) == bad
    assert q(P(), 64, 4, 60, None, 0, P(), 64, P(), 2, None) == uns
    assert q(P(), 64, 4, 64, P(), 0, P(), 64, P(), 2, None) == bad
    assert q(P(), 56, 4, 64, None, 0, P(), 64, P(), 2, None) == bad
    assert q(P(), 68, 4, 64, None, 0, P(), 64, P(), 2, None) == uns
    assert q(P(), 64, 4, 64, None, 0, P(), 56, P(), 2, None) == bad
    assert q(P(), 64, 4, 64, None, 0, P(), 68, P(), 2, None) == uns
    assert q(P(), 64, 4, 64, None, 0, P(), 64, P(), 1, None) == bad
    assert q(None, 64, 4, 64, None, 0, P(), 64, P(), 2, None) == bad
    assert q(P(4104), 64, 4, 64, None, 0, P(), 64, P(), 2, None) == uns
    assert q(None, 64, 0, 64, None, 0, None, 64, None, 2, None) == L.MOE_OK
    d = L.LIB.moe_act8_dequantize
    assert d(P(), 64, P(), 2, 4, 64, None, 0, P(), 56, None) == bad
    assert d(P(), 64, P(), 2, 4, 64, None, 0, None, 64, None) == bad
    f = L.LIB.moe_act8_swiglu_fwd
    assert f(P(), 120, 4, 64, None, 0, P(), 64, P(), 128, P(), 4, None) == bad
    assert f(P(), 128, 4, 64, None, 0, P(), 56, P(), 128, P(), 4, None) == bad
    assert f(P(), 128, 4, 64, None, 0, P(), 64, P(), 64, P(), 4, None) == bad
    assert f(P(), 128, 4, 64, None, 0, P(), 64, P(), 128, P(), 3, None) == bad
    assert f(P(), 128, 4, 64, None, 0, P(4100), 64, P(), 128, P(), 4, None) == uns
    b = L.LIB.moe_act8_swiglu_bwd
    assert b(P(), 128, P(), 4, P(), 56, 4, 64, None, 0, P(), 128, None, 0, None) == bad
    assert b(P(), 128, P(), 4, P(), 64, 4, 64, None, 0, P(), 120, None, 0, None) == bad
    assert b(P(), 128, P(), 4, P(), 64, 4, 64, None, 0, P(), 128, P(), 8, None) == bad
    assert b(P(), 128, P(), 4, P(), 64, 4, 64, None, 0, None, 128, None, 0, None) == bad
    assert b(P(), 128, P(), 4, P(), 64, 4, 64, None, 0, P(), 128, P(4100), 64, None) == uns


def test_unknown_format_name(L):
    from mixture_experts_grouped_router_gb300 import lowbit
    with pytest.raises(ValueError, match="MXFP4"):
        lowbit.Fp4Rows(4, 64, 1, "fp4", device="cpu")
