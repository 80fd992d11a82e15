"""The products with an epilogue, y = act(W x' + b) * mul + r, against the
same formula in 64 bits on the oracle's product.

Tolerances.  The sums s of the products differ from the oracle's by at most
ds = 2e-3 max |s| of the token's row (the products' own bar).  With v = s +
bias, |act'| <= 1.13 (SILU 1.10, both GELUs 1.13) and, for RELU2, 2 |v| + ds,
the epilogue in fp32 is off by at most ds |act'| |mul| and about ten roundings
and function errors, 2^-20 of (|v| |mul| + |r|) in all (RELU2: v^2 |mul|), and
y by half an fp16 step, 2^-11 |y| (at least 2^-25)."""
import itertools

import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg
from gpu_helpers import gen_matrix, oracle_y

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FMTS = ("PQ2_0", "PTQ1_0", "Q1_0", "Q2_0_G64")
ACTS = tuple(bgg.ACTIVATIONS)


def erf(x):
    return torch.erf(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def act64(v, name):
    if name == "relu":
        return np.where(v < 0, 0, v)
    if name == "relu2":
        return np.where(v < 0, 0, v) ** 2
    if name == "silu":
        with np.errstate(over="ignore"):
            return v / (1 + np.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + erf(v / np.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    return v


class Case:
    def __init__(self, fmt, N, K, M, seed=3, which="bmr", pad=0, scale=1.0):
        self.fmt, self.N, self.K, self.M = fmt, N, K, M
        T, S = gen_matrix(seed, 0, N, K, fmt=fmt)
        rng = np.random.default_rng(seed)
        self.x = (rng.standard_normal((M, K)) * scale).astype(np.float16)
        self.s = np.asarray(oracle_y(fmt, T, S, self.x))
        self.d = bgg.bgg_describe(fmt, N, K)
        self.packed = bgg.upload(bgg.bgg_pack_weights(self.d, T, S))
        size = float(np.std(self.s)) or 1.0

        def operand(shape, sc):
            a = np.zeros((shape[0], shape[1] + pad), np.float16)
            a[:, :shape[1]] = rng.standard_normal(shape) * sc
            return a[:, :shape[1]], torch.from_numpy(a).cuda()[:, :shape[1]]

        self.b = (rng.standard_normal(N) * size).astype(np.float16) if "b" in which else None
        self.mul, self.mul_d = operand((M, N), 1.0) if "m" in which else (None, None)
        self.r, self.r_d = operand((M, N), size) if "r" in which else (None, None)
        self.b_d = None if self.b is None else torch.from_numpy(self.b).cuda()
        self.x_d = torch.from_numpy(self.x).cuda()

    def want(self, act):
        """(y, tolerance) in 64 bits."""
        ds = 2e-3 * np.abs(self.s).max(axis=1, keepdims=True)
        v = self.s + (0 if self.b is None else self.b.astype(np.float64))
        mul = 1.0 if self.mul is None else self.mul.astype(np.float64)
        r = 0.0 if self.r is None else self.r.astype(np.float64)
        y = act64(v, act) * mul + r
        slope = 2 * np.abs(v) + ds if act == "relu2" else 1.13
        size = (v * v if act == "relu2" else np.abs(v)) * np.abs(mul) + np.abs(r)
        off = ds * slope * np.abs(mul) + 2.0 ** -20 * size
        return y, off + 2.0 ** -11 * (np.abs(y) + off) + 2.0 ** -25

    def run(self, act, how="call", ws=None, y=None, **change):
        kw = dict(dict(activation=act, bias=self.b_d, mul=self.mul_d, residual=self.r_d), **change)
        gemv = how != "gemm"
        if y is None:
            y = torch.full((self.M, self.N), float("nan"), dtype=torch.float16, device="cuda")
        if ws is None:
            size = (bgg.bgg_gemv_workspace_size if gemv else bgg.bgg_gemm_workspace_size)(self.d, self.M)
            ws = bgg.workspace(size)
        rot = bgg.BGG_ROTATE_INPUT
        if how == "call":
            bgg.bgg_ternary_gemv_epilogue(self.d, self.packed, self.x_d, y, self.M, rot, ws, **kw)
        elif how == "gemm":
            bgg.bgg_ternary_gemm_epilogue(self.d, self.packed, self.x_d, y, self.M, rot, ws, **kw)
        else:
            bgg.bgg_gemv_prepare(self.d, self.x_d, self.M, rot, ws)
            bgg.bgg_gemv_run_epilogue(self.d, self.packed, y, self.M, ws, **kw)
        torch.cuda.synchronize()
        return y

    def check(self, y, act):
        want, tol = self.want(act)
        y = y.double().cpu().numpy()
        fits = np.abs(want) + tol < 65504
        bad = ~(np.abs(y - want) <= tol) & fits
        assert not bad.any(), (act, np.argwhere(bad)[:4], y[bad][:4], want[bad][:4], tol[bad][:4])
        assert np.all(fits | (np.abs(y) >= 65000) | (np.abs(y - want) <= tol))


# every decode kernel family: one launch and two steps, split and unsplit K
@pytest.mark.parametrize("fmt,M", [(f, m) for f in FMTS for m in (1, 2, 3, 4, 5, 16)])
@pytest.mark.parametrize("N,K", [(100, 640), (256, 5120), (9000, 256)])
def test_gemv_formats_and_tokens(fmt, M, N, K):
    c = Case(fmt, N, K, M)
    c.check(c.run("silu"), "silu")
    c.check(c.run("none", how="steps"), "none")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("which", ["", "b", "m", "r", "bm", "br", "mr", "bmr"])
def test_every_activation_and_operand(act, which):
    for fmt, M in (("PQ2_0", 1), ("PTQ1_0", 6)):
        c = Case(fmt, 320, 1280, M, which=which)
        c.check(c.run(act), act)
    c = Case("PQ2_0", 320, 1280, 40, which=which)
    c.check(c.run(act, how="gemm"), act)


@pytest.mark.parametrize("fmt", ["PQ2_0", "PTQ1_0"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (17, 100, 640), (77, 6100, 1280), (130, 1001, 256), (512, 320, 384),
                                   (300, 17408, 256), (640, 5120, 512), (129, 8, 128), (127, 264, 256)])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_gemm_sizes(fmt, M, N, K, pad):
    """Unsplit and split K, ragged tiles, rows of operands on 16 bytes and
    off them."""
    c = Case(fmt, N, K, M, pad=pad)
    c.check(c.run("gelu", how="gemm"), "gelu")
    x = torch.empty((M, K), dtype=torch.float16, device="cuda")
    bgg.bgg_hadamard_rotate(c.x_d, x, M, K)
    for act in ("relu", "silu"):
        guard = torch.full((M * N + 512,), 7.0, dtype=torch.float16, device="cuda")
        y = guard[256:256 + M * N].view(M, N)
        y.fill_(float("nan"))
        bgg.bgg_ternary_gemm_epilogue(c.d, c.packed, x, y, M, 0, None, activation=act, bias=c.b_d, mul=c.mul_d,
                                      residual=c.r_d)  # no workspace: unsplit, PTQ1_0 without the rewrite
        torch.cuda.synchronize()
        c.check(y, act)
        assert torch.all(guard[:256] == 7.0) and torch.all(guard[-256:] == 7.0)


@pytest.mark.parametrize("fmt", ["PQ2_0", "PTQ1_0"])
@pytest.mark.parametrize("M", [17, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128])
def test_prompts_of_one_tile(fmt, M):
    """Every height of the product's tile, split with an epilogue and unsplit
    without; a token's sums do not depend on how many come with it."""
    N, K = 333, 1408
    c = Case(fmt, N, K, M)
    c.check(c.run("silu", how="gemm"), "silu")
    # the same tokens and more, K in one range in both: PQ2_0 without a
    # workspace, PTQ1_0 with one that holds the weights rewritten and no more
    ws = None if fmt == "PQ2_0" else bgg.workspace(c.d.row_tiles * 64 * K // 4)
    more = torch.cat([c.x_d, torch.zeros((128 - M, K), dtype=torch.float16, device="cuda")])
    got = []
    for x in (c.x_d, more):
        guard = torch.full((len(x) * N + 512,), 7.0, dtype=torch.float16, device="cuda")
        y = guard[256:256 + len(x) * N].view(len(x), N)
        y.fill_(float("nan"))
        bgg.bgg_ternary_gemm(c.d, c.packed, x, y, len(x), 0, ws)
        torch.cuda.synchronize()
        assert torch.all(guard[:256] == 7.0) and torch.all(guard[-256:] == 7.0)
        got.append(y[:M])
    assert torch.equal(*got)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("which", ["b", "m", "r", "bmr"])
def test_wide_rows_with_every_activation(act, which):
    """Unsplit prompt products whose operands are all on 16 bytes."""
    c = Case("PQ2_0", 520, 256, 140, which=which)
    x = torch.empty((140, 256), dtype=torch.float16, device="cuda")
    bgg.bgg_hadamard_rotate(c.x_d, x, 140, 256)
    y = torch.full((140, 520), float("nan"), dtype=torch.float16, device="cuda")
    bgg.bgg_ternary_gemm_epilogue(c.d, c.packed, x, y, 140, 0, None, activation=act, bias=c.b_d, mul=c.mul_d,
                                  residual=c.r_d)
    c.check(y, act)
    # the same values a value at a time (y off 16 bytes)
    odd = torch.full((140 * 520 + 1,), float("nan"), dtype=torch.float16, device="cuda")[1:].view(140, 520)
    bgg.bgg_ternary_gemm_epilogue(c.d, c.packed, x, odd, 140, 0, None, activation=act, bias=c.b_d, mul=c.mul_d,
                                  residual=c.r_d)
    assert torch.equal(odd, y)


def test_large_sums_pass_the_activations():
    """Pre-activations far on both sides: exponentials that overflow and
    vanish."""
    for act in ACTS:
        c = Case("PQ2_0", 128, 2560, 2, which="b", scale=200.0)
        c.check(c.run(act), act)


@pytest.mark.parametrize("how,M", [("call", 1), ("call", 7), ("steps", 1), ("gemm", 33)])
@pytest.mark.parametrize("fmt", ["PQ2_0", "PTQ1_0"])
def test_y_as_residual_or_multiplier(fmt, how, M):
    """In place: the residual stream, and the up projection's buffer."""
    for N, K in ((300, 17408), (5000, 512)):  # split and unsplit K
        c = Case(fmt, N, K, M)
        apart = c.run("none", how=how, mul=None)
        y = c.r_d.clone()
        assert torch.equal(c.run("none", how=how, y=y, mul=None, residual=y), apart)
        apart = c.run("silu", how=how, residual=None)
        y = c.mul_d.clone()
        assert torch.equal(c.run("silu", how=how, y=y, mul=y, residual=None), apart)
        y = c.mul_d.clone()
        both = c.run("gelu", how=how, mul=c.mul_d, residual=c.mul_d)
        assert torch.equal(c.run("gelu", how=how, y=y, mul=y, residual=y), both)


def test_nothing_asked_is_the_product():
    for fmt, M, how in itertools.product(("PQ2_0", "PTQ1_0"), (1, 3, 9, 50), ("call", "gemm")):
        if how == "call" and M > 16:
            continue
        c = Case(fmt, 700, 1280, M, which="")
        y = torch.empty((M, 700), dtype=torch.float16, device="cuda")
        ws = bgg.workspace(max(bgg.bgg_gemm_workspace_size(c.d, M), bgg.bgg_gemv_workspace_size(c.d, min(M, 16))))
        (bgg.bgg_ternary_gemv if how == "call" else bgg.bgg_ternary_gemm)(c.d, c.packed, c.x_d, y, M, 1, ws)
        assert torch.equal(c.run("none", how=how), y)


@pytest.mark.parametrize("fmt,M", [("PQ2_0", 1), ("PQ2_0", 3), ("PQ2_0", 9), ("PTQ1_0", 1), ("PTQ1_0", 5), ("Q1_0", 2)])
def test_nan_passes_every_activation(fmt, M):
    for N, K in ((200, 5120), (8000, 256)):
        c = Case(fmt, N, K, M, which="m")
        c.x_d[M - 1, 7] = float("nan")
        for act in ACTS:
            y = c.run(act)
            assert torch.isnan(y[M - 1]).all()
            assert torch.isfinite(y[:M - 1]).all()


def test_infinite_operands():
    c = Case("PQ2_0", 128, 256, 2)
    c.b_d[3], c.b_d[4] = float("inf"), float("-inf")
    c.r_d[:, 9] = float("nan")
    c.mul_d[:, :] = c.mul_d.abs() + 0.5
    y = c.run("relu")
    assert torch.all(y[:, 3] == float("inf")) and torch.isnan(y[:, 9]).all()
    assert torch.equal(y[:, 4], c.r_d[:, 4])  # relu(-inf) = 0
    y = c.run("silu")
    assert torch.all(y[:, 3] == float("inf"))


def test_workspace_and_tokens_stay_apart():
    """Row words are zero after an epilogue call, and a token's row does not
    depend on the others."""
    c = Case("PQ2_0", 192, 17408, 4)
    ws = bgg.workspace(bgg.bgg_gemv_workspace_size(c.d, 16))
    y = c.run("silu", ws=ws)
    assert not ws[:16 << 20].any()
    for m in range(4):
        one = torch.empty((1, 192), dtype=torch.float16, device="cuda")
        bgg.bgg_ternary_gemv_epilogue(c.d, c.packed, c.x_d[m:m + 1].contiguous(), one, 1, 1, ws, activation="silu",
                                      bias=c.b_d, mul=c.mul_d[m:m + 1], residual=c.r_d[m:m + 1])
        assert torch.equal(one[0], y[m])


def test_graph_replays():
    for how, M, K in (("call", 1, 17408), ("call", 12, 5120), ("gemm", 70, 5120)):
        c = Case("PTQ1_0", 640, K, M)
        want = c.run("silu", how=how)
        y = torch.zeros_like(want)
        ws = bgg.workspace(max(bgg.bgg_gemv_workspace_size(c.d, min(M, 16)), bgg.bgg_gemm_workspace_size(c.d, M)))
        call = bgg.bgg_ternary_gemv_epilogue if how == "call" else bgg.bgg_ternary_gemm_epilogue
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            call(c.d, c.packed, c.x_d, y, M, 1, ws, activation="silu", bias=c.b_d, mul=c.mul_d, residual=c.r_d)
        torch.cuda.synchronize()
        for _ in range(3):
            y.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_rows_beyond_one_launch():
    """65600 rows: two launches of split tiles."""
    c = Case("PQ2_0", 65600, 5120 * 2, 1, which="br")
    c.check(c.run("silu"), "silu")


def test_binding_refusals():
    c = Case("PQ2_0", 128, 256, 3)
    for change in (dict(bias=c.b_d[:-1]), dict(bias=c.b_d.float()), dict(mul=c.mul_d[:, ::2]), dict(mul=c.mul_d[:2]),
                   dict(residual=c.r_d.t()), dict(residual=c.r_d.cpu()), dict(mul=c.mul_d.float())):
        with pytest.raises(ValueError):
            c.run("silu", **change)
    with pytest.raises(KeyError):
        c.run("swish")
    with pytest.raises(bgg.BggError) as e:
        c.run(17)
    assert e.value.status == 2
    wide = torch.zeros((3, 136), dtype=torch.float16, device="cuda")
    with pytest.raises(bgg.BggError) as e:  # y as an operand of another stride
        y = wide.view(-1)[:3 * 128].view(3, 128)
        c.run("silu", y=y, residual=wide[:, :128])
    assert e.value.status == 3
