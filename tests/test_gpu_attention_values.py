"""Attention over caches with extreme values: NaN and infinities where
every score is -inf."""
import math

import pytest

import bit_gemv_gemm_amd as bgg  # noqa: F401
from test_gpu_attention import Device, case

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
