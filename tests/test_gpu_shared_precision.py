"""The probabilities of a shared prefix enter their product with the values as
bgg_paged_attention's do, as a sum of two 16-bit terms.

Tolerance: test_gpu_attention's (2^-16 sum p |v| for the two terms), and where
the values are fp16 or E4M3 (multiplied as fp16) 2^-32 sum |v| / sum p more, with
the row's largest p one: a probability below 2^-21 of it has no second term, and
its first one is off by half of fp16's smallest step, 2^-25, after the lift of
2^7.  Values of both signs make every element small next to sum p |v|, so that
the rounding of the output itself hides nothing: one term alone is off by up to
2^-8 (bf16) or 2^-11 (fp16) of that sum."""
import math

import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg
from test_gpu_attention import TYPES
from test_gpu_shared_attention import Device, case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def check(c, out, lse):
    """out [B, hq, D] and lse [B, hq] against the formula in 64 bits."""
    hq, hk, D, page = c["hq"], c["hk"], c["D"], c["page"]
    q = c["q"].double().numpy().reshape(len(c["lengths"]), hq, D)
    eps = torch.finfo(TYPES[c["dtype"]]).eps / 2
    for b, n in enumerate(c["lengths"]):
        t = np.arange(n)
        pg, t = torch.from_numpy(c["full"][b].numpy()[t // page]).long(), torch.from_numpy(t % page).long()
        for h in range(hq):
            kh = h // (hq // hk)
            k, v = (x[pg, kh, t].double().numpy() for x in c["caches"])
            if c["scales"][0] is not None:
                k, v = k * float(c["scales"][0][kh]), v * float(c["scales"][1][kh])
            s = k @ q[b, h] * c["scale"]
            size = (np.abs(k) @ np.abs(q[b, h])).max() * abs(c["scale"])
            p = np.exp(s - s.max())
            l = p.sum()
            o, x = p @ v / l, s.max() + math.log(l)
            e = 2 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -20
            tol = eps * np.abs(o) + (e + 2.0 ** -16 + n * 2.0 ** -23) * (p @ np.abs(v) / l) + 2.0 ** -25
            if c["kv"] != "bf16":
                tol = tol + 2.0 ** -32 * np.abs(v).sum(0) / l
            bad = ~(np.abs(out[b, h] - o) <= tol)
            assert not bad.any(), (b, h, np.argwhere(bad)[:5].ravel(), out[b, h][bad][:5], o[bad][:5], tol[bad][:5])
            assert abs(lse[b, h] - x) <= e + n * 2.0 ** -23 + 2.0 ** -22 * abs(x), (b, h, lse[b, h], x)


def run_check(c, both=False):
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    B = len(c["lengths"])
    check(c, d.out.double().cpu().numpy().reshape(B, c["hq"], c["D"]), d.lse.double().cpu().numpy())
    if both:
        bgg.bgg_paged_attention(d.d, d.k, d.v, c["full"].cuda(), d.n, d.q, d.out, d.ws, scale=c["scale"], lse=d.lse,
                                k_scale=d.ks, v_scale=d.vs)
        torch.cuda.synchronize()
        check(c, d.out.double().cpu().numpy().reshape(B, c["hq"], c["D"]), d.lse.double().cpu().numpy())


KINDS = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]


@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("D,hq,hk", [(64, 8, 1), (96, 6, 2), (128, 12, 2), (192, 3, 3), (256, 4, 1)])
def test_two_terms(dtype, kv, D, hq, hk):
    """Tokens of two scores per head, their values of opposite signs; a prefix
    that ends inside a tile."""
    c = case([(11, [1, 20, 3])], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=16, seed=D)
    k, v = c["caches"]
    up = torch.zeros(k.shape[0], k.shape[2], dtype=torch.bool)
    for p in range(k.shape[0]):
        up[p, p % 3::2] = True
    wide = 100.0 if kv == "e4m3" else 1.0
    one = torch.where(up[:, None, :, None], wide, -wide)
    c["caches"] = [(one * torch.linspace(0.01, 0.05, D)).to(k.dtype).expand(k.shape).contiguous(),
                   (one * torch.linspace(0.5, 2.0, D)).to(v.dtype).expand(v.shape).contiguous()]
    run_check(c)


@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("D,hq,hk", [(64, 4, 1), (128, 6, 2), (256, 3, 1)])
def test_spread_scores(dtype, kv, D, hq, hk):
    run_check(case([(40, [1, 30, 200]), (3, [5])], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=32, seed=D, spread=2.0),
              both=True)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("D,hq,hk", [(64, 16, 1), (128, 12, 2), (192, 3, 3), (256, 4, 1)])
@pytest.mark.parametrize("window", [0, 6000])
def test_infinite_values_in_a_long_prefix(kv, D, hq, hk, window):
    """In several chunks, behind which every row sees the whole chunk or, with
    a window, some rows a part: the sums of such values are formed once for the
    former."""
    c = case([(130, [1, 70, 40, 500])], hq=hq, hk=hk, D=D, page=64, dtype="bf16" if kv == "bf16" else "f16", kv=kv,
             window=window, seed=D)
    inf, nan = float("inf"), float("nan")
    planted = [(7, {5000: nan}), (D - 1, {8319: nan}), (20, {2500: nan})]  # (a window's start lies between 2321 and 2820)
    if kv != "e4m3":
        planted += [(8, {5000: inf}), (9, {4100: -inf, 8000: -inf}), (10, {100: inf, 7000: -inf}), (11, {0: inf, 2400: inf}),
                    (12, {2600: inf})]
    v, clean = c["caches"][1].clone(), c["caches"][1].clone()
    for dim, tokens in planted:
        for t, x in tokens.items():
            v[int(c["full"][0, t // 64]), :, t % 64, dim], clean[int(c["full"][0, t // 64]), :, t % 64, dim] = x, 0.0
    got, want = Device(dict(c, caches=[c["caches"][0], v])), Device(dict(c, caches=[c["caches"][0], clean]))
    got.step(), want.step()
    torch.cuda.synchronize()
    B = len(c["lengths"])
    out, ref = got.out.view(B, hq, D), want.out.view(B, hq, D).clone()
    for b, n in enumerate(c["lengths"]):
        for dim, tokens in planted:
            x = sum(x for t, x in tokens.items() if t >= (max(0, n - window) if window else 0))
            if x != 0:
                ref[b, :, dim] = x
    assert torch.equal(got.lse, want.lse)
    same = (out == ref) | (torch.isnan(out) & torch.isnan(ref))
    assert same.all(), (~same).nonzero()[:8]


@pytest.mark.parametrize("dtype,kv", KINDS)
@pytest.mark.parametrize("gap", [10, 16, 21, 24, 27, 31])
def test_a_first_token_that_takes_nearly_all(dtype, kv, gap):
    """Its values are zero, and every other token's probability is 2^-gap of its
    own: the elements are sums of small probabilities alone.  The stated bound,
    2^-32 of the largest probability a token for fp16 and E4M3 values, is all
    that separates them from 0 at the end of the range."""
    D, hq, hk = 64, 4, 1
    c = case([(125, [1, 30, 200])], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=16, seed=gap)
    k, v = torch.zeros(c["caches"][0].shape), c["caches"][1].float().abs()
    first = int(c["full"][0, 0])
    k[first, :, 0, 0] = 256.0  # (exact in every type)
    v[first, :, 0] = 0.0
    c["caches"] = [k.to(TYPES[kv]), v.to(TYPES[kv])]
    c["q"] = torch.zeros_like(c["q"])
    c["q"].view(-1, hq, D)[:, :, 0] = 8.0
    c["scale"] = gap * math.log(2) / (8.0 * 256.0 * (float(c["scales"][0][0]) if kv == "e4m3" else 1.0))
    run_check(c, both=True)
