"""Rotary positions of tokens with several positions (time, height, width)
against the formula in 64 bits; tolerances as for one position per token
(test_gpu_rotary.py)."""
import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg
from test_gpu_rotary import TYPES, case, check, check_case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def axes_case(sections, arrangement="blocks", pos_pad=0, **kw):
    """A case of test_gpu_rotary whose positions are [A, T] and whose
    rotated part is the sections'."""
    c = case(R=2 * sum(sections), **kw)
    g = torch.Generator().manual_seed(kw.get("seed", 1) + 100)
    far = kw.get("far", 5000)
    c["pos3"] = torch.randint(-far if kw.get("neg") else 0, far + 1, (len(sections), c["T"] + pos_pad), generator=g,
                              dtype=torch.int32)[:, :c["T"]]
    c["axes"] = torch.from_numpy(bgg.bgg_rotary_axes(sections, arrangement))
    return c


def run(c, cache=True, in_place=False, stream=None):
    dev = "cuda"
    nq, nk = c["hq"] * c["D"], c["hk"] * c["D"]
    row = c["row"].to(dev)
    q, k, v = row[:, :nq], row[:, nq:nq + nk], row[:, nq + nk:nq + 2 * nk]
    out = q if in_place else torch.full((c["T"], nq), float("nan"), dtype=TYPES[c["dtype"]], device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    ks, vs = (None if x is None else x.to(dev) for x in c["scales"])
    d = bgg.bgg_cache_describe(c["kv"], c["pages"], c["page"], c["hk"], c["D"])
    base = c["pos3"].storage_offset(), c["pos3"].stride(0)
    # (the same strides on the device)
    whole = torch.full((c["pos3"].shape[0], max(base[1], 1)), 99, dtype=torch.int32, device=dev)
    pos = whole[:, :c["T"]]
    pos.copy_(c["pos3"])
    if not cache:
        bgg.bgg_rotary_append_axes(d, None, None, pos, c["axes"].to(dev), None, c["freqs"].to(dev), q=q, q_out=out,
                                   layout=c["layout"], magnitude=c["mag"], stream=stream)
    else:
        bgg.bgg_rotary_append_axes(d, kc, vc, pos, c["axes"].to(dev), c["slots"].to(dev), c["freqs"].to(dev), q=q, q_out=out,
                                   k=k, v=v, layout=c["layout"], magnitude=c["mag"], k_scale=ks, v_scale=vs, stream=stream)
    torch.cuda.synchronize()
    return out, kc, vc


def check_axes(c, got, monkeypatch):
    """check_case with the angle of each pair from its own axis."""
    import test_gpu_rotary

    def rotated(x, pos, freqs, layout, mag):
        R = 2 * len(freqs)
        a = (c["pos3"].numpy()[c["axes"].numpy()].astype(np.float64) * freqs.astype(np.float64)[:, None]).T[:, None, :]
        cos, sin = np.cos(a), np.sin(a)
        y, size = x.copy(), np.zeros_like(x)
        i = np.arange(R // 2)
        iu, iw = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
        u, w = x[..., iu], x[..., iw]
        y[..., iu], y[..., iw] = mag * (u * cos - w * sin), mag * (u * sin + w * cos)
        size[..., iu] = size[..., iw] = mag * (np.abs(u) + np.abs(w))
        return y, size

    monkeypatch.setattr(test_gpu_rotary, "rotated", rotated)
    check_case(c, *got)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D,sections,arrangement", [
    (64, [32], "blocks"), (128, [16, 24, 24], "blocks"), (128, [24, 20, 20], "cyclic"), (96, [1, 2, 9], "blocks"),
    (256, [11, 11, 10], "cyclic"), (192, [0, 40, 0, 7], "blocks"), (64, [3, 2, 2], "cyclic"), (256, [64, 64], "blocks")])
def test_every_type_layout_and_arrangement(layout, dtype, kv, D, sections, arrangement, monkeypatch):
    c = axes_case(sections, arrangement, D=D, layout=layout, dtype=dtype, kv=kv, mag=1.25)
    check_axes(c, run(c), monkeypatch)


@pytest.mark.parametrize("T,hq,hk,page,pad,pos_pad", [(1, 1, 1, 16, 0, 0), (1, 48, 8, 64, 0, 5), (2, 7, 1, 32, 8, 1),
                                                      (300, 32, 32, 16, 0, 77), (1000, 5, 5, 64, 8, 0)])
def test_sizes_and_strides(T, hq, hk, page, pad, pos_pad, monkeypatch):
    c = axes_case([8, 12, 12], T=T, hq=hq, hk=hk, page=page, pad=pad, D=64, dtype="bf16", kv="bf16", seed=T, pos_pad=pos_pad)
    check_axes(c, run(c), monkeypatch)


@pytest.mark.parametrize("neg", [False, True])
def test_far_positions_in_place(neg, monkeypatch):
    c = axes_case([16, 24, 24], T=40, far=2**31 - 1, neg=neg, seed=3)
    check_axes(c, run(c, in_place=True), monkeypatch)


@pytest.mark.parametrize("sections,layout", [([16, 16], "half"), ([16, 16], "interleaved"), ([5, 6, 20], "half")])
def test_queries_without_a_cache(sections, layout, monkeypatch):
    c = axes_case(sections, T=77, hq=12, D=64, layout=layout, dtype="bf16", kv="e4m3")
    out, _, _ = run(c, cache=False)
    x = c["row"][:, :12 * 64].double().numpy().reshape(77, 12, 64)
    a = (c["pos3"].numpy()[c["axes"].numpy()].astype(np.float64) * c["freqs"].numpy().astype(np.float64)[:, None]).T[:, None]
    n = sum(sections)
    i = np.arange(n)
    iu, iw = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    want, size = x.copy(), np.zeros_like(x)
    u, w = x[..., iu], x[..., iw]
    want[..., iu], want[..., iw] = u * np.cos(a) - w * np.sin(a), u * np.sin(a) + w * np.cos(a)
    size[..., iu] = size[..., iw] = np.abs(u) + np.abs(w)
    check(out.double().cpu().numpy().reshape(77, 12, 64), want, size, "bf16")


@pytest.mark.parametrize("R", [64, 44])
def test_one_position_on_every_axis_is_the_plain_call(R):
    """The same bits as bgg_rotary_append, with the row expanded (stride 0),
    repeated, or as the only axis."""
    c = case(T=50, D=64, R=R, hq=4, hk=4, seed=9)
    dev = "cuda"
    row, pos, freqs, slots = c["row"].to(dev), c["pos"].to(dev), c["freqs"].to(dev), c["slots"].to(dev)
    d = bgg.bgg_cache_describe("f16", c["pages"], c["page"], 4, 64)
    axes = (torch.arange(R // 2, device=dev) % 3).to(torch.uint8)

    def go(call, *a):
        out, kc, vc = torch.zeros((50, 256), dtype=torch.float16, device=dev), *(x.to(dev) for x in c["caches"])
        call(d, kc, vc, *a, slots, freqs, q=row[:, :256], q_out=out, k=row[:, 256:512], v=row[:, 512:768])
        return out, kc, vc

    want = go(bgg.bgg_rotary_append, pos)
    for p, a in ((pos.expand(3, 50), axes), (pos.repeat(3, 1), axes), (pos[None], torch.zeros_like(axes)),
                 (pos.repeat(4, 1), torch.full_like(axes, 200))):  # (an axis past the last is the last)
        for x, y in zip(go(bgg.bgg_rotary_append_axes, p, a), want):
            assert torch.equal(x, y)


def test_captured_call(monkeypatch):
    c = axes_case([16, 24, 24], T=9, seed=2)
    dev = "cuda"
    nq, nk = c["hq"] * c["D"], c["hk"] * c["D"]
    row = c["row"].to(dev)
    out = torch.zeros((9, nq), dtype=torch.float16, device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    start = kc.clone(), vc.clone()
    pos, ax, sl, fr = c["pos3"].contiguous().to(dev), c["axes"].to(dev), c["slots"].to(dev), c["freqs"].to(dev)
    d = bgg.bgg_cache_describe("f16", c["pages"], c["page"], c["hk"], c["D"])

    def go():
        bgg.bgg_rotary_append_axes(d, kc, vc, pos, ax, sl, fr, q=row[:, :nq], q_out=out, k=row[:, nq:nq + nk],
                                   v=row[:, nq + nk:nq + 2 * nk])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        go()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            go()
    for i in range(4):
        c["pos3"] = torch.randint(0, 90000, (3, 9), dtype=torch.int32)
        pos.copy_(c["pos3"])
        kc.copy_(start[0]), vc.copy_(start[1])
        graph.replay()
        torch.cuda.synchronize()
        check_axes(c, (out, kc, vc), monkeypatch)


def test_refusals_of_the_binding():
    dev = "cuda"
    d = bgg.bgg_cache_describe("f16", 2, 16, 1, 64)
    q = torch.zeros((3, 64), dtype=torch.float16, device=dev)
    pos, ax = torch.zeros((2, 3), dtype=torch.int32, device=dev), torch.zeros(32, dtype=torch.uint8, device=dev)
    fr = torch.ones(32, device=dev)
    bgg.bgg_rotary_append_axes(d, None, None, pos, ax, None, fr, q=q, q_out=q)
    for p, a, f in ((pos[0], ax, fr), (pos.long(), ax, fr), (pos.t(), ax, fr), (pos, ax[:5], fr), (pos, ax.int(), fr),
                    (pos, None, fr), (pos.cpu(), ax, fr), (pos[:, :2], ax, fr),
                    (torch.zeros((3, 2), dtype=torch.int32, device=dev).t(), ax, fr)):
        with pytest.raises((ValueError, bgg.BggError)):
            bgg.bgg_rotary_append_axes(d, None, None, p, a, None, f, q=q, q_out=q)
    with pytest.raises(bgg.BggError):
        bgg.bgg_rotary_append_axes(d, None, None, torch.zeros((5, 3), dtype=torch.int32, device=dev), ax, None, fr, q=q, q_out=q)
    bgg.bgg_rotary_append_axes(d, None, None, pos[:, :0], ax, None, fr, q=q[:0], q_out=q[:0])
