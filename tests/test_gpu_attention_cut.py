"""Attention over sequences that are cut into chunks and joined: every head
dimension with each way the join shares its columns out, more parts than a
thread has in flight, windows that begin inside a chunk's first tile, 8-bit
caches; and a decode step of a layer whose sequences are cut, on every cache
type.  Tolerances as in test_gpu_attention."""
import pytest

import bit_gemv_gemm_amd as bgg
from test_gpu_attention import Device, case, run_check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# heads of 96, 192 and 256: 24, 48 and 64 columns of four values per query
# head, on 256 threads (1, 2, 3, 6 and 16 heads: ten threads per column to
# four columns per thread)
@pytest.mark.parametrize("dtype,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [96, 192, 256])
@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (6, 2), (6, 1), (16, 1), (17, 1)])
def test_joins_of_every_head_dimension(dtype, kv, D, hq, hk):
    run_check(case([2900, 40, 777], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=32, seed=D + hq))


@pytest.mark.parametrize("D,hq", [(64, 1), (96, 1), (96, 5), (128, 2), (192, 3), (256, 1), (256, 9)])
def test_many_parts(D, hq):
    """About 60 parts: several rounds of the loads that a thread has in
    flight, more than sixteen maxima per head."""
    run_check(case([31001], hq=hq, hk=1, D=D, page=128, seed=D))


@pytest.mark.parametrize("D,kv,hq,hk", [(64, "f16", 8, 8), (96, "e4m3", 4, 2), (128, "f16", 12, 2), (192, "f16", 2, 1),
                                        (256, "e4m3", 6, 1), (256, "f16", 24, 4)])
@pytest.mark.parametrize("window", [513, 545, 1000, 2047, 2900])
def test_windows_of_several_chunks(D, kv, hq, hk, window):
    """The first visible token anywhere in its tile and page; what lies before
    the window is NaN, or on pages that the table no longer has."""
    lengths = [3000, 2999, 2048, 700, 513]
    c = case(lengths, hq=hq, hk=hk, D=D, kv=kv, page=64, window=window, seed=window)
    for b, n in enumerate(lengths):
        first = max(0, n - window)
        for x in c["caches"]:
            for pg in range(-(-first // 64)):
                x[c["table"][b, pg], :, :min(64, first - 64 * pg)] = float("nan")
        if b % 2 == 0:
            c["table"][b, :first // 64] = -1
    run_check(c)


def test_pages_outside_the_cache_in_a_cut_sequence():
    """Whole chunks whose pages are hidden, and single pages within chunks."""
    c = case([6000, 3100], hq=6, hk=1, D=96, page=16, seed=6)
    c["table"][0, 3] = c["table"][0, 200] = -1
    c["table"][0, 60:180] = c["pages"]
    c["table"][1, :150] = -5
    run_check(c)


@pytest.mark.parametrize("D", [96, 192, 256])
def test_cut_sequences_again_and_as_a_graph(D):
    c = case([5000, 800, 3], hq=8, hk=2, D=D, dtype="bf16", kv="bf16", page=64, seed=D)
    a = run_check(c)
    first, lse = a.out.clone(), a.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        a.step()
    torch.cuda.synchronize()
    for _ in range(4):
        a.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, first) and torch.equal(a.lse, lse)
        a.step()
        torch.cuda.synchronize()
        assert torch.equal(a.out, first)


@pytest.mark.parametrize("D,kv", [(96, "f16"), (128, "e4m3"), (256, "bf16")])
def test_queries_replaced_by_their_outputs(D, kv):
    """out may be q itself."""
    dtype = "bf16" if kv == "bf16" else "f16"
    c = case([3000, 1, 70, 0, 900], hq=40, hk=2, D=D, dtype=dtype, kv=kv, page=32, seed=D)
    a = run_check(c)
    b = Device(c)
    b.out = b.q
    b.step()
    torch.cuda.synchronize()
    assert torch.equal(b.q, a.out) and torch.equal(b.lse, a.lse)


# --- appending to a cache and attending over it, sequences cut ---------------
@pytest.mark.parametrize("kv,dtype", [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("layout,D,R", [("half", 96, 64), ("interleaved", 128, 128)])
def test_prompt_then_decode_steps(kv, dtype, layout, D, R):
    """A prompt's keys and values appended at once, then decode steps (append
    and attention in a row, no wait between them) in which the sequences pass
    the length from which they are cut.  The attention is checked over what
    the cache holds, and the cache against the rotated rows."""
    hq, hk, page, start, steps = 6, 2, 16, (505, 0, 1700), 9
    tt = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
    B, g = len(start), torch.Generator().manual_seed(D)
    width = -(-(max(start) + steps) // page)
    pages = B * width + 1
    d = bgg.bgg_cache_describe(kv, pages, page, hk, D)
    cache = [torch.zeros((pages, hk, page, D), dtype=tt[kv], device="cuda") for _ in range(2)]
    scale = [torch.tensor([0.02, 0.03]) * (i + 1) if kv == "e4m3" else None for i in range(2)]
    dscale = [None if s is None else s.cuda() for s in scale]
    table = (torch.randperm(pages - 1, generator=g)[:B * width].view(B, width) + 1).int()
    freqs, mag = bgg.bgg_rotary_frequencies(R, 10000.0, "parts", 4.0, trained_length=512.0)
    fr = torch.from_numpy(freqs).cuda()
    nq, nk = hq * D, hk * D

    def slots(b, t):
        return table[b, t // page].long() * page + t % page

    def append(row, pos, sl, q_out):
        bgg.bgg_rotary_append(d, *cache, pos.int().cuda(), sl.cuda(), fr, q=row[:, :nq], q_out=q_out, k=row[:, nq:nq + nk],
                              v=row[:, nq + nk:], layout=layout, magnitude=mag, k_scale=dscale[0], v_scale=dscale[1])

    rows = []  # (sequence, token, host row)
    for b, n in enumerate(start):
        if n:
            t = torch.arange(n)
            row = torch.randn((n, nq + 2 * nk), generator=g).to(tt[dtype])
            append(row.cuda(), t, slots(b, t), torch.empty((n, nq), dtype=tt[dtype], device="cuda"))
            rows.append((b, t, row))
    ws = bgg.workspace(bgg.bgg_attention_workspace_size(d, hq, B))
    seen = []
    for i in range(steps):
        t = torch.tensor(start) + i
        row = torch.randn((B, nq + 2 * nk), generator=g).to(tt[dtype])
        q = torch.empty((B, nq), dtype=tt[dtype], device="cuda")
        out, lse = torch.empty_like(q), torch.empty((B, hq), device="cuda")
        lengths = (t + 1).int().cuda()
        append(row.cuda(), t, torch.stack([slots(b, t[b]) for b in range(B)]), q)
        bgg.bgg_paged_attention(d, *cache, table.cuda(), lengths, q, out, ws, scale=D ** -0.5, lse=lse, k_scale=dscale[0],
                                v_scale=dscale[1])
        seen.append((t, q, out, lse))
        for b in range(B):
            rows.append((b, t[b:b + 1], row[b:b + 1]))
    torch.cuda.synchronize()
    host = [x.cpu() for x in cache]
    # the cache: every row at its slot (values exact but for their one
    # rounding, keys rotated; bounds of the rotary tests, twice over)
    half = torch.finfo(tt[kv]).eps / 2
    for b, t, row in rows:
        z = row.double().view(len(t), hq + 2 * hk, D)
        ang = t.double()[:, None, None] * torch.from_numpy(freqs).double()
        iu = torch.arange(R // 2) * (1 if layout == "half" else 2)
        iw = iu + (R // 2 if layout == "half" else 1)
        k, v = z[:, hq:hq + hk].clone(), z[:, hq + hk:]
        u, w = k[..., iu].clone(), k[..., iw].clone()
        k[..., iu] = mag * (u * ang.cos() - w * ang.sin())
        k[..., iw] = mag * (u * ang.sin() + w * ang.cos())
        pg, cell = table[b, t // page].long(), t % page
        for x, want, s in ((host[0], k, scale[0]), (host[1], v, scale[1])):
            got = x[pg, :, cell].double()
            sc = torch.ones(hk, 1, dtype=torch.float64) if s is None else s.double()[:, None]
            assert torch.all((got * sc - want).abs() <= 2 * half * want.abs() + 2.0 ** -9 * (sc if s is not None else 0)
                             + 2.0 ** -18 * 8)
    # the attention, over the cache as it was then: later tokens lie past each length
    for t, q, out, lse in seen:
        c = dict(lengths=(t + 1).tolist(), hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=page, window=0, pages=pages,
                 table=table, caches=host, scales=scale, q=q.cpu(), scale=D ** -0.5)
        have = Device.__new__(Device)
        have.c, have.out, have.lse = c, out, lse
        have.check()
    assert not ws[:16384].any()


def test_a_batch_changes_bits_but_not_the_result():
    """The chunks follow all lengths of a call, so the same sequence beside
    others may round differently; it stays within the same bounds."""
    c = case([2500, 90], hq=6, hk=2, D=128, page=64, seed=3)
    alone = dict(c, lengths=c["lengths"][:1], table=c["table"][:1], q=c["q"][:1])
    more = dict(c, lengths=c["lengths"] + [2400] * 6, table=c["table"][[0, 1] + [0] * 6].contiguous(),
                q=torch.cat([c["q"], c["q"][:1].repeat(6, 1)]))
    for x in (alone, c, more):
        run_check(x)
