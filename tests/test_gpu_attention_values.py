"""Attention over caches with extreme values: infinities at visible tokens,
NaN and infinities where every score is -inf, and bfloat16 values near both
ends of its range.
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


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,hq,hk", [(64, 2, 1), (96, 6, 2), (128, 12, 1), (192, 3, 3), (256, 16, 1)])
@pytest.mark.parametrize("page", [16, 128])
def test_infinite_values_of_visible_tokens(dtype, D, hq, hk, page):
    """An infinite value makes its element infinite, NaN where both signs or
    a NaN meet; nothing else changes.  Sequence 1 is cut into several chunks."""
    lengths = [40, 2100, 1]
    c = case(lengths, hq=hq, hk=hk, D=D, dtype=dtype, kv=dtype, page=page, seed=D)
    c["q"] = c["q"].abs() + 0.5
    for t in (20, 900):  # a token of sequence 1 and one of 0 with a probability of zero
        put(c, 0, int(t > 40), t, slice(None), -300.0)
    planted = [  # sequence, dimension, {token: value}, element
        (0, 5, {3: INF}, INF), (0, 6, {39: -INF}, -INF), (0, 7, {0: INF, 30: INF}, INF), (0, 8, {1: INF, 2: -INF}, NAN),
        (0, 9, {1: INF, 25: NAN}, NAN), (0, 10, {20: -INF}, -INF), (0, D - 1, {17: INF}, INF),
        (1, 0, {0: INF}, INF), (1, 5, {2099: -INF}, -INF), (1, 6, {10: INF, 1500: INF}, INF),
        (1, 7, {10: INF, 1500: -INF}, NAN), (1, 8, {900: INF}, INF), (1, 9, {900: INF, 2000: NAN}, NAN),
        (1, 11, {1024: -INF}, -INF), (2, 4, {0: INF}, INF), (2, D - 2, {0: NAN}, NAN)]
    clean = dict(c, caches=[x.clone() for x in c["caches"]])
    for b, dim, tokens, _ in planted:
        for t, v in tokens.items():
            put(c, 1, b, t, dim, v)
            put(clean, 1, b, t, dim, 0.0)
    out, lse = result(c)
    want, wlse = result(clean)
    for b, dim, _, v in planted:
        want[b, :, dim] = v
    assert torch.equal(lse, wlse)
    same = (out == want) | (torch.isnan(out) & torch.isnan(want))
    assert same.all(), [(tuple(i), float(out[tuple(i)]), float(want[tuple(i)])) for i in (~same).nonzero()[:6].tolist()]


def test_an_infinite_value_where_the_maximum_rises():
    """The token with the infinite value loses all its weight to a later one
    of the same wave, of another wave, of another chunk."""
    c = case([1, 300, 4000], hq=4, hk=1, D=64, page=64, seed=3)
    c["q"] = c["q"].abs() + 0.5
    put(c, 1, 1, 2, 7, INF)
    put(c, 1, 2, 2, 8, -INF)
    for b, t in ((1, 2 + 128), (2, 3900)):
        put(c, 0, b, t, slice(None), 300.0)
    put(c, 1, 1, 200, 9, INF)
    out, _ = result(c)
    assert (out[1, :, 7] == INF).all() and (out[1, :, 9] == INF).all() and (out[2, :, 8] == -INF).all()
    rest = out.clone()
    rest[1, :, 7] = rest[1, :, 9] = rest[2, :, 8] = 0
    assert torch.isfinite(rest).all()


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
