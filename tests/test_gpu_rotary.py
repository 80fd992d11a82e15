"""Rotary positions and the append to the paged cache against the formula in
64 bits.

Tolerances.  The kernel rotates in fp32: the angle is exact to one fp32
rounding of a value of at most pi (2^-24 pi < 1.9e-7), sin and cos to two
units (2^-22), each product and the sum to half a unit, so a rotated value is
within 8e-7 magnitude (|u| + |w|) of the formula, plus half a step of the
stored type: eps/2 of the value (for fp16 at least 2^-25, for e4m3 2^-10 of
its scale, the half steps below their normal ranges)."""
import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
FLOOR = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10}
SLACK = 8e-7


def half_eps(t):
    return torch.finfo(TYPES[t]).eps / 2


def rotated(x, pos, freqs, layout, mag):
    """x float64 [T, H, D]; (rotated, |u| + |w| of each value's pair, 0 past
    the rotated part)."""
    R = 2 * len(freqs)
    a = pos.astype(np.float64)[:, None, None] * freqs.astype(np.float64)
    c, s = np.cos(a), np.sin(a)
    y, size = x.copy(), np.zeros_like(x)
    i = np.arange(R // 2)
    iu, iw = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
    u, w = x[..., iu], x[..., iw]
    y[..., iu], y[..., iw] = mag * (u * c - w * s), mag * (u * s + w * c)
    size[..., iu] = size[..., iw] = mag * (np.abs(u) + np.abs(w))
    return y, size


def check(got, want, size, t, scale=1.0):
    """got, want: values (a cache's with their scale applied)."""
    tol = half_eps(t) * (np.abs(want) + SLACK * size) + FLOOR[t] * scale + SLACK * (size + (np.abs(want) if t == "e4m3" else 0))
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def case(T=5, hq=6, hk=2, D=128, R=128, layout="half", dtype="f16", kv="f16", page=16, mag=1.0, far=5000, seed=1,
         pad=0, neg=False):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    row = torch.randn((T, (hq + 2 * hk) * D + pad), generator=g).to(dt)
    pages = -(-T // page) + 2
    cells = (torch.randperm(pages, generator=g)[:, None] * page + torch.arange(page)).reshape(-1)
    slots = cells[torch.randperm(len(cells), generator=g)[:T]].clone()
    if T > 3:
        slots[1], slots[T - 1] = -1, pages * page  # outside the cache on both sides
    pos = torch.randint(-far if neg else 0, far + 1, (T,), generator=g, dtype=torch.int32)
    freqs = torch.from_numpy(bgg.bgg_rotary_frequencies(R, 10000.0)[0])
    caches = [(torch.randn((pages, hk, page, D), generator=g) * 3).to(TYPES[kv]) for _ in range(2)]
    scales = [torch.rand((hk,), generator=g) * 0.02 + 0.005 if kv == "e4m3" else None for _ in range(2)]
    return dict(T=T, hq=hq, hk=hk, D=D, R=R, layout=layout, dtype=dtype, kv=kv, page=page, mag=mag, row=row, slots=slots,
                pos=pos, freqs=freqs, caches=caches, scales=scales, pages=pages)


def run(c, stream=None, in_place=False):
    """(q_out, k cache, v cache) on the device."""
    dev = "cuda"
    nq, nk = c["hq"] * c["D"], c["hk"] * c["D"]
    row = c["row"].to(dev)
    q, k, v = row[:, :nq], row[:, nq:nq + nk], row[:, nq + nk:nq + 2 * nk]
    out = q if in_place else torch.full((c["T"], nq), float("nan"), dtype=TYPES[c["dtype"]], device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    ks, vs = (None if x is None else x.to(dev) for x in c["scales"])
    d = bgg.bgg_cache_describe(c["kv"], c["pages"], c["page"], c["hk"], c["D"])
    bgg.bgg_rotary_append(d, kc, vc, c["pos"].to(dev), c["slots"].to(dev), c["freqs"].to(dev), q=q, q_out=out, k=k, v=v,
                          layout=c["layout"], magnitude=c["mag"], k_scale=ks, v_scale=vs, stream=stream)
    torch.cuda.synchronize()
    return out, kc, vc


def check_case(c, q_out, kc, vc):
    T, hq, hk, D = c["T"], c["hq"], c["hk"], c["D"]
    x = c["row"][:, :(hq + 2 * hk) * D].double().numpy().reshape(T, hq + 2 * hk, D)
    pos, freqs, mag = c["pos"].numpy(), c["freqs"].numpy(), float(np.float32(c["mag"]))
    want, size = rotated(x[:, :hq], pos, freqs, c["layout"], mag)
    check(q_out.double().cpu().numpy().reshape(T, hq, D), want, size, c["dtype"])
    kw, ksize = rotated(x[:, hq:hq + hk], pos, freqs, c["layout"], mag)
    vw, vsize = x[:, hq + hk:], np.zeros_like(x[:, hq + hk:])
    slots = c["slots"].numpy()
    for cache, start, want, size, scale in ((kc, c["caches"][0], kw, ksize, c["scales"][0]),
                                            (vc, c["caches"][1], vw, vsize, c["scales"][1])):
        got = cache.cpu().transpose(1, 2).reshape(-1, hk, D)
        first = start.transpose(1, 2).reshape(-1, hk, D)
        touched = np.zeros(len(got), dtype=bool)
        for t, s in enumerate(slots):
            if not 0 <= s < len(got):
                continue
            touched[s] = True
            sc = np.ones(hk) if scale is None else scale.double().numpy()
            w = np.clip(want[t], -448 * sc[:, None], 448 * sc[:, None]) if scale is not None else want[t]
            check(got[s].double().numpy() * sc[:, None], w, size[t], c["kv"], sc[:, None])
        bits = torch.uint8 if c["kv"] == "e4m3" else torch.int16
        assert torch.equal(got.contiguous().view(bits)[~touched], first.contiguous().view(bits)[~touched])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D,R", [(64, 64), (96, 48), (128, 128), (192, 64), (256, 256), (256, 2), (128, 126), (64, 12)])
def test_every_type_and_layout(layout, dtype, kv, D, R):
    c = case(D=D, R=R, layout=layout, dtype=dtype, kv=kv, mag=1.25)
    check_case(c, *run(c))


@pytest.mark.parametrize("T,hq,hk,page,pad", [(1, 1, 1, 16, 0), (1, 48, 8, 64, 0), (2, 7, 1, 32, 8), (17, 24, 4, 256, 40),
                                              (300, 32, 32, 16, 0), (1000, 5, 5, 64, 8)])
def test_sizes_and_strides(T, hq, hk, page, pad):
    c = case(T=T, hq=hq, hk=hk, page=page, pad=pad, D=64, R=64, dtype="bf16", kv="bf16", seed=T)
    check_case(c, *run(c))


@pytest.mark.parametrize("far", [1 << 18, 1 << 24, (1 << 31) - 1])
def test_far_and_negative_positions(far):
    """The angle of a far position is formed in 64 bits: float32 products
    would be off by up to 2^31 * 2^-24 = 128 turns."""
    c = case(T=9, far=far, neg=True, seed=3)
    c["pos"][0], c["pos"][1], c["pos"][2] = far, -far, 0
    c["slots"][1] = 3 if 3 not in c["slots"].tolist() else c["slots"][1]
    check_case(c, *run(c))


@pytest.mark.parametrize("T,hq,hk,layout", [(2, 4096, 1024, "half"), (20001, 2, 1, "interleaved"), (1, 1, 1024, "half")])
def test_many_heads_and_tokens(T, hq, hk, layout):
    c = case(T=T, hq=hq, hk=hk, D=64, R=32, layout=layout, seed=T)
    check_case(c, *run(c))


def test_in_place_queries():
    c = case(T=20, seed=5)
    check_case(c, *run(c, in_place=True))


def test_queries_or_keys_alone():
    c = case(T=6, seed=8)
    dev, nq, nk = "cuda", c["hq"] * c["D"], c["hk"] * c["D"]
    whole, kc0, vc0 = run(c)
    d = bgg.bgg_cache_describe("f16", c["pages"], c["page"], c["hk"], c["D"])
    row, out = c["row"].to(dev), torch.empty((c["T"], c["hq"], c["D"]), dtype=torch.float16, device=dev)
    pos, slots, freqs = c["pos"].to(dev), c["slots"].to(dev), c["freqs"].to(dev)
    bgg.bgg_rotary_append(d, None, None, pos, None, freqs, q=row[:, :nq].view(c["T"], c["hq"], c["D"]), q_out=out,
                          layout="half")
    assert torch.equal(out.view(c["T"], nq), whole)
    kc, vc = (x.to(dev) for x in c["caches"])
    bgg.bgg_rotary_append(d, kc, vc, pos, slots, freqs, k=row[:, nq:nq + nk], v=row[:, nq + nk:], layout="half")
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_e4m3_cut_nan_and_inf():
    c = case(T=2, hq=1, hk=1, D=64, R=2, kv="e4m3", far=0, seed=2)
    c["scales"] = [torch.tensor([0.5]), torch.tensor([2.0])]
    c["row"][0, 64 + 8:64 + 12] = torch.tensor([1000.0, -1000.0, float("inf"), float("nan")])
    c["row"][0, 128:128 + 4] = torch.tensor([1000.0, -1000.0, float("-inf"), float("nan")])
    _, kc, vc = run(c)
    s = int(c["slots"][0])
    k = kc[s // c["page"], 0, s % c["page"]].float().cpu()
    v = vc[s // c["page"], 0, s % c["page"]].float().cpu()
    assert k[8] == 448 and k[9] == -448 and k[10] == 448 and torch.isnan(k[11])
    assert v[0] == 448 and v[1] == -448 and v[2] == -448 and torch.isnan(v[3])


def test_e4m3_every_value_rounds_to_nearest():
    """Every finite e4m3 value, the midpoints between neighbours and the fp16
    values beside the midpoints, at scale 1 and position 0."""
    vals = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mid, torch.nextafter(mid.half(), torch.tensor(1e4).half()).float(),
                   torch.nextafter(mid.half(), torch.tensor(0.0).half()).float()])
    x = torch.cat([x, -x])
    T = -(-len(x) // 64)
    flat = torch.zeros(T * 64)
    flat[:len(x)] = x
    c = case(T=T, hq=1, hk=1, D=64, R=2, kv="e4m3", far=0)
    c["slots"] = torch.arange(T)
    c["scales"] = [torch.ones(1), torch.ones(1)]
    c["row"][:, 128:] = flat.view(T, 64).half()
    _, _, vc = run(c)
    got = vc.view(-1, 64)[:T].float().cpu().view(-1)
    assert torch.equal(got, flat.half().float().to(torch.float8_e4m3fn).float())


def test_offsets_past_32_bits():
    """Slots whose byte and value offsets pass 2^32 and 2^31."""
    hk, page, D = 8, 64, 256
    pages = (1 << 31) // (hk * page * D) + 40  # 2^31 values and more
    d = bgg.bgg_cache_describe("f16", pages, page, hk, D)
    assert d.total_bytes > 1 << 32
    kc = torch.empty((pages, hk, page, D), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    T = 3
    slots = torch.tensor([pages * page - 1, (pages - 20) * page + 5, 0], device="cuda")
    x = torch.randn((T, 2, hk, D), device="cuda").half()
    kc.view(-1)[:: 1 << 22] = 7
    bgg.bgg_rotary_append(d, kc, vc, torch.zeros(T, dtype=torch.int32, device="cuda"), slots,
                          torch.ones(1, device="cuda"), k=x[:, 0].reshape(T, -1), v=x[:, 1].reshape(T, -1))
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, :, s % page], x[t, 0])
        assert torch.equal(vc[s // page, :, s % page], x[t, 1])


def test_graph_replays_on_a_side_stream():
    c = case(T=40, seed=11)
    want = run(c)
    dev, nq, nk = "cuda", c["hq"] * c["D"], c["hk"] * c["D"]
    d = bgg.bgg_cache_describe("f16", c["pages"], c["page"], c["hk"], c["D"])
    row, pos, slots, freqs = c["row"].to(dev), c["pos"].to(dev), c["slots"].to(dev), c["freqs"].to(dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    out = torch.zeros((c["T"], nq), dtype=torch.float16, device=dev)

    def step():
        bgg.bgg_rotary_append(d, kc, vc, pos, slots, freqs, q=row[:, :nq], q_out=out, k=row[:, nq:nq + nk],
                              v=row[:, nq + nk:], layout="half")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            step()
    for _ in range(3):
        out.zero_()
        kc.copy_(c["caches"][0])
        vc.copy_(c["caches"][1])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(kc, want[1]) and torch.equal(vc, want[2])


def test_binding_refusals():
    c = case(T=4)
    dev, nq, nk = "cuda", c["hq"] * c["D"], c["hk"] * c["D"]
    d = bgg.bgg_cache_describe("f16", c["pages"], c["page"], c["hk"], c["D"])
    row, pos, slots, freqs = c["row"].to(dev), c["pos"].to(dev), c["slots"].to(dev), c["freqs"].to(dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    q, k, v = row[:, :nq], row[:, nq:nq + nk], row[:, nq + nk:]
    good = dict(q=q, q_out=torch.empty_like(q), k=k, v=v)
    a = (d, kc, vc, pos, slots, freqs)
    for change in (dict(q_out=torch.empty((3, nq), dtype=torch.float16, device=dev)), dict(k=k[:, :-1]), dict(k=k.float()),
                   dict(v=v.cpu()), dict(v=None), dict(k_scale=freqs.double()), dict(q_out=torch.empty_like(q)[:, ::2])):
        with pytest.raises(ValueError):
            bgg.bgg_rotary_append(*a, **dict(good, **change))
    with pytest.raises(ValueError):
        bgg.bgg_rotary_append(d, kc[1:], vc, pos, slots, freqs, **good)
    with pytest.raises(ValueError):
        bgg.bgg_rotary_append(d, kc, vc, pos.long(), slots, freqs, **good)
    with pytest.raises(ValueError):
        bgg.bgg_rotary_append(d, kc, vc, pos, slots.int(), freqs, **good)
    with pytest.raises(bgg.BggError):
        bgg.bgg_rotary_append(d, kc, vc, pos, slots, torch.ones(65, device=dev), **good)
    with pytest.raises(bgg.BggError):
        bgg.bgg_rotary_append(*a, **dict(good, k=row[:, nq + 4:nq + nk + 4]))  # rows off 16 bytes
    none = dict(q=q[:0], q_out=torch.empty_like(q[:0]), k=k[:0], v=v[:0])
    bgg.bgg_rotary_append(d, kc, vc, pos[:0], slots[:0], freqs, **none)
    torch.cuda.synchronize()
