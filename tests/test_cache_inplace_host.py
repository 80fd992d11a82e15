"""Attention with its output in the place of the queries: one stride, or the
call is refused (before anything is enqueued, so no GPU is needed)."""
import ctypes

import pytest

import bit_gemv_gemm_amd as bgg
from test_cache_host import ATTENTION, LIB, P, SHAPE, describe


def attention(**change):
    return LIB.bgg_paged_attention(ctypes.byref(describe()), bgg._ATTENTION_ARGS.pack(*dict(ATTENTION, **change).values()),
                                   None)


@pytest.mark.parametrize("change", [dict(qs=256, os=512), dict(qs=512, os=256)])
def test_two_strides_in_place_are_refused(change):
    assert attention(out=P, **change) == SHAPE


@pytest.mark.parametrize("change", [dict(batch=0), dict(batch=0, out=P + 4096, os=512)])
def test_allowed(change):
    assert attention(**change) == 0
