"""The products' epilogue alone, y = act(s + bias) * mul + residual: inputs
whose sums s are known exactly (small whole activations that are not rotated,
scales that are powers of two; every partial sum is a multiple of 2^-13 and
below 2^11, so fp32 adds them without rounding), so that only the epilogue's
own error is allowed.  Half of the residuals are minus the rounded rest of
the formula: what is left is below half an fp16 step of it, and any rounding
to fp16 on the way shows.

Tolerance.  With v = s + bias (one rounding, 2^-24 |v|, times a slope of at
most 1.13) the functions are off by, relative to |v|: RELU nothing; SILU, and
GELU_TANH alike: exponential, sum, reciprocal and product 1 + 1/2 + 1 + 1/2
units of 2^-23 of a factor below one, the exponent's own roundings at most a
third of a unit more (p (1 - p) |exponent| <= 0.31); GELU: erfc to 4 units,
its argument to 1.5 * 2^-24 times a slope below 1/2, two products.  All are
below 2^-21 |v|; RELU2 is off by 3 * 2^-24 v^2.  The multiplier and the
residual add two roundings, so the fp32 value is within
e = 2^-20 (|v| |mul| + |r|) (RELU2: v^2 |mul|), and y within
e + 2^-11 (|y| + e) + 2^-25, one rounding to fp16."""
import functools

import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg
import synth

torch = pytest.importorskip("torch")

ACTS = tuple(bgg.ACTIVATIONS)
UNIT = 2.0 ** -13

# (how, format, tokens, rows, K, workspace): every kernel that has an epilogue
CASES = [
    # one launch: one token, two to four
    *[("call", "PQ2_0", m, n, k, True) for m in (1, 2, 4) for n, k in ((100, 17408), (9000, 256), (130, 128))],
    *[("call", "PTQ1_0", m, n, k, True) for m in (1, 2) for n, k in ((100, 17408), (9000, 256), (130, 128))],
    # two launches, matrix cores
    *[("call", f, m, n, k, True) for f, m in (("PQ2_0", 5), ("PQ2_0", 16), ("PTQ1_0", 3), ("PTQ1_0", 16), ("Q1_0", 1),
                                              ("Q1_0", 16), ("Q2_0_G64", 1), ("Q2_0_G64", 9))
      for n, k in ((100, 5120), (4500, 256))],
    # prepared activations, one token
    *[("steps", f, 1, n, k, True) for f in ("PQ2_0", "PTQ1_0") for n, k in ((100, 5120), (4500, 256))],
    # prompts, K in one range: short tiles, values at a time, 16 bytes at a time, PTQ1_0 as it is
    *[("gemm", "PQ2_0", m, n, 256, False) for m, n in ((20, 136), (60, 131), (90, 136), (140, 131), (140, 136))],
    ("gemm", "PTQ1_0", 140, 136, 320 * 4, False), ("gemm", "PTQ1_0", 33, 131, 640, False),
    # K in several ranges: eight, four and one value per thread of the adding kernel
    *[("gemm", f, m, n, 5120, True) for f, m, n in (("PQ2_0", 20, 136), ("PQ2_0", 60, 132), ("PTQ1_0", 90, 131),
                                                    ("PQ2_0", 300, 136), ("PTQ1_0", 200, 132))],
]


def erf(x):
    return torch.erf(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def act64(v, name):
    if name == "relu":
        return np.where(v < 0, 0, v)
    if name == "relu2":
        return np.where(v < 0, 0, v) ** 2
    if name == "silu":
        return v / (1 + np.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + erf(v / np.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    return v


def f16(a):
    return a.astype(np.float16).astype(np.float64)


class Sums:
    """Weights, activations and their sums s [M, N], exact."""

    def __init__(self, how, fmt, M, N, K):
        self.fmt, self.M, self.N, self.K = fmt, M, N, K
        rng = np.random.default_rng([M, N, K])
        self.T = synth.weights(fmt, 7, 0, N, K)
        group = synth.scale_group(fmt)
        S = rng.integers(1, 3, (N, K // group))  # scales of one or two units
        self.S = (S * UNIT).astype(np.float16)
        most = int(np.clip(16384 / (0.58 * np.sqrt(0.62 * K)), 1, 2047))
        x = rng.integers(-most, most + 1, (M, K))
        self.x = x.astype(np.float16)
        assert np.array_equal(self.x.astype(np.int64), x)
        assert K * most * 2 <= 2 ** 24  # units that any partial sum has at most
        s = x.astype(np.float64) @ (self.T.astype(np.float64) * np.repeat(S, group, axis=1)).T
        self.s = s * UNIT
        self.bias = f16(rng.standard_normal(N))
        self.mul = f16(rng.standard_normal((M, N)) + np.where(rng.random((M, N)) < 0.5, 1, -1))
        self.noise = f16(3 * rng.standard_normal((M, N)))


@functools.lru_cache(maxsize=2)
def sums(how, fmt, M, N, K):
    return Sums(how, fmt, M, N, K)


class Epilogue:
    """Operands over those sums.  which: 'all' (bias, multiplier, a random
    residual), 'rest' (the residual takes the rounded rest away), 'sum' (no
    bias or multiplier; the residual takes the rounded act(s) away)."""

    def __init__(self, c, act, which):
        self.c, self.act, self.which = c, act, which
        self.bias, self.mul = (None, None) if which == "sum" else (c.bias, c.mul)
        self.r = c.noise if which == "all" else -f16(self.formula(0.0))

    def formula(self, r, bias=None, mul=None, act=None, after=lambda v, step: v):
        b = 0.0 if self.bias is None else self.bias
        m = 1.0 if self.mul is None else self.mul
        v = after(after(self.c.s, "sum") + b, "bias")
        return after(after(act64(v, act or self.act), "activation") * m, "multiplier") + r

    def refused(self, y):
        """Where y (float64) is further off than the epilogue may be."""
        v = np.abs(self.c.s + (0.0 if self.bias is None else self.bias))
        m = 1.0 if self.mul is None else np.abs(self.mul)
        want = self.formula(self.r)
        e = 2.0 ** -20 * ((v * v if self.act == "relu2" else v) * m + np.abs(self.r))
        return ~(np.abs(y - want) <= e + 2.0 ** -11 * (np.abs(want) + e) + 2.0 ** -25)


WHICH = ("all", "rest", "sum")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("case", [("call", "PQ2_0", 1, 130, 128), ("call", "Q1_0", 1, 100, 5120), ("gemm", "PQ2_0", 20, 136, 256),
                                  ("call", "PTQ1_0", 2, 100, 17408)], ids=str)
def test_the_check_refuses_wrong_epilogues(case, act):
    """On the CPU: the formula rounded once passes, and each planted mistake
    is refused, at the smallest of the cases too."""
    c = sums(*case)
    assert np.abs(c.s).max() > 3 and np.mean(f16(c.s) != c.s) > 0.3  # sums that fp16 does not hold
    for which in WHICH:
        e = Epilogue(c, act, which)
        assert not e.refused(f16(e.formula(e.r))).any()
        if act in ("gelu", "gelu_tanh", "silu"):
            for other in ("gelu", "gelu_tanh", "silu", "relu"):
                if other != act:
                    assert e.refused(f16(e.formula(e.r, act=other))).any(), (which, other)
        if which == "all":
            continue
        for at in ("sum", "bias", "activation", "multiplier"):
            wrong = e.formula(e.r, after=lambda v, step: f16(v) if step == at else v)
            assert e.refused(f16(wrong)).any(), (which, at)
    e = Epilogue(c, act, "all")
    v = c.s + c.bias
    wrong = [act64(v, act) * (c.mul + e.r), (act64(v, act) + e.r) * c.mul, act64(c.s, act) + c.bias * c.mul + e.r,
             act64(c.s, act) * c.mul + e.r]
    if act != "none":
        wrong += [act64(v * c.mul, act) + e.r, (act64(c.s, act) + c.bias) * c.mul + e.r]
    for y in wrong:
        assert e.refused(f16(y)).any()


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_epilogue_on_exact_sums(case):
    how, fmt, M, N, K, with_ws = case
    c = sums(*case[:5])
    d = bgg.bgg_describe(fmt, N, K)
    packed = bgg.upload(bgg.bgg_pack_weights(d, c.T, c.S))
    x = torch.from_numpy(c.x).cuda()

    def up(a):
        return None if a is None else torch.from_numpy(a.astype(np.float16)).cuda()

    size = (bgg.bgg_gemm_workspace_size if how == "gemm" else bgg.bgg_gemv_workspace_size)(d, M)
    ws = bgg.workspace(size) if with_ws else None
    for act in ACTS:
        for which in WHICH:
            e = Epilogue(c, act, which)
            y = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
            kw = dict(activation=act, bias=up(e.bias), mul=up(e.mul), residual=up(e.r))
            if how == "call":
                bgg.bgg_ternary_gemv_epilogue(d, packed, x, y, M, 0, ws, **kw)
            elif how == "gemm":
                bgg.bgg_ternary_gemm_epilogue(d, packed, x, y, M, 0, ws, **kw)
            else:
                bgg.bgg_gemv_prepare(d, x, M, 0, ws)
                bgg.bgg_gemv_run_epilogue(d, packed, y, M, ws, **kw)
            torch.cuda.synchronize()
            got = y.double().cpu().numpy()
            bad = e.refused(got)
            want = e.formula(e.r)
            assert not bad.any(), (act, which, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
            if act == "none" and which == "sum":  # s - fp16(s) is a fp16 value
                assert np.array_equal(got, want)
