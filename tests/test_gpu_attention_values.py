"""Attention over caches with extreme values: NaN and infinities where
every score is -inf, and bfloat16 values near both ends of its range.
Tolerances as in test_gpu_attention."""
import math

import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg  # noqa: F401
from test_gpu_attention import Device, case, formula

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def put(c, which, b, t, dim, value):
    """Cache `which` (0 keys, 1 values) of sequence b, token t."""
    page = int(c["table"][b, t // c["page"]])
    c["caches"][which][page, :, t % c["page"], dim] = value


def result(c):
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    shape = (len(c["lengths"]), c["hq"], c["D"])
    return d.out.view(shape).clone(), d.lse.clone()


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_no_score_but_minus_infinity(dtype, value):
    """Every score -inf: out is 0 and lse -inf, whatever the values are (one
    chunk, and several)."""
    c = case([50, 1500, 33], hq=2, hk=1, D=64, dtype=dtype, kv=dtype, seed=12)
    c["q"][:] = 1.0
    for b, n in ((0, 50), (1, 1500)):
        for t in range(n):
            put(c, 0, b, t, slice(None), -INF)
            put(c, 1, b, t, slice(None), value)
    out, lse = result(c)
    assert not out[:2].any() and torch.all(lse[:2] == -math.inf)
    assert torch.isfinite(out[2]).all() and torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("power", [120, 112, -100])
@pytest.mark.parametrize("D,hq,hk", [(64, 4, 1), (128, 6, 2), (256, 16, 1)])
def test_bfloat16_values_near_the_ends_of_its_range(power, D, hq, hk):
    c = case([1, 40, 1500], hq=hq, hk=hk, D=D, dtype="bf16", kv="bf16", seed=D)
    # out is linear in the values, and bfloat16 holds them times 2^power
    # exactly: the formula and its tolerance of the values as they were, times
    # 2^power (2^-25, half a step of fp16's subnormals, has no part in this)
    want, wlse, tol, ltol = formula(c)
    c["caches"][1].mul_(2.0 ** power)
    out, lse = result(c)
    assert np.all(np.abs(out.double().cpu().numpy() * 2.0 ** -power - want) <= tol - 2.0 ** -25)
    assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= ltol)


def test_one_largest_bfloat16_value():
    """A single token's value comes out as it is, the largest finite one too."""
    top = torch.finfo(torch.bfloat16).max
    c = case([1, 1], hq=2, hk=1, D=64, dtype="bf16", kv="bf16", seed=5)
    put(c, 1, 0, 0, slice(None), top)
    put(c, 1, 1, 0, slice(None), torch.finfo(torch.bfloat16).smallest_normal)
    out, _ = result(c)
    assert torch.all(out[0] == top) and torch.all(out[1] == torch.finfo(torch.bfloat16).smallest_normal)
