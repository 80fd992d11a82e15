"""Refusals of the products with an epilogue: all before anything is
enqueued, so they need no GPU."""
import ctypes

import pytest

import bit_gemv_gemm_amd as bgg

LIB = ctypes.CDLL(bgg.LIB_PATH)
P = 1 << 20  # stands for a device pointer; no refused call touches it
NULL, FORMAT, SHAPE, BUFFER, DESC = 1, 2, 3, 6, 7
GOOD = dict(act=3, reserved=0, bias=P, mul=P, residual=P, ms=256, rs=300)


def call(which, d, ep, x=P, packed=P, y=P + 4096, M=2, flags=1, ws=P, wsb=1 << 30):
    vp, i64, u32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
    e = None if ep is None else bgg._EPILOGUE.pack(*ep.values())
    d = None if d is None else ctypes.byref(d)
    if which == "run":
        return LIB.bgg_gemv_run_epilogue(d, vp(packed), vp(y), i64(M), e, vp(ws), sz(wsb), None)
    f = LIB.bgg_ternary_gemv_epilogue if which == "gemv" else LIB.bgg_ternary_gemm_epilogue
    return f(d, vp(packed), vp(x), vp(y), i64(M), u32(flags), e, vp(ws), sz(wsb), None)


@pytest.mark.parametrize("which", ["gemv", "run", "gemm"])
@pytest.mark.parametrize("change,status", [
    (dict(act=-1), FORMAT), (dict(act=6), FORMAT), (dict(reserved=1), SHAPE), (dict(bias=P + 1), BUFFER),
    (dict(mul=P + 1), BUFFER), (dict(residual=P + 1), BUFFER), (dict(ms=255), SHAPE), (dict(rs=-300), SHAPE),
    (dict(ms=1 << 41), SHAPE), (dict(mul=0), SHAPE), (dict(residual=0), SHAPE), (dict(mul=P + 4096, ms=300), SHAPE),
    (dict(residual=P + 4096), SHAPE)])
def test_epilogue_refusals(which, change, status):
    d = bgg.bgg_describe("PQ2_0", 256, 512)
    assert call(which, d, dict(GOOD, **change)) == status


@pytest.mark.parametrize("which", ["gemv", "run", "gemm"])
def test_other_refusals_as_without_epilogue(which):
    d = bgg.bgg_describe("PQ2_0", 256, 512)
    assert call(which, d, None) == NULL
    assert call(which, None, GOOD) == NULL
    assert call(which, d, GOOD, packed=None) == NULL
    assert call(which, d, GOOD, y=None) == NULL
    assert call(which, d, GOOD, M=0) == SHAPE
    assert call(which, d, GOOD, packed=P + 8) == BUFFER
    if which != "gemm":
        assert call(which, d, GOOD, M=17) == SHAPE
        assert call(which, d, GOOD, wsb=64) == BUFFER
        assert call(which, d, GOOD, ws=None) == NULL
    else:
        assert call(which, bgg.bgg_describe("Q1_0", 256, 512), GOOD) == FORMAT
    if which != "run":
        assert call(which, d, GOOD, x=None) == NULL
        assert call(which, d, GOOD, flags=2) == SHAPE
    d.K += 128
    assert call(which, d, GOOD) == DESC
