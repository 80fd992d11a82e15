"""Attention of one new token over the paged cache against the formula in 64
bits.

Tolerances.  A score's fp32 sum of D products is within (D + 8) 2^-24
|scale| sum |q k| of the exact one; with S the largest |scale| sum |q k| of
a row, every probability is within a factor 1 +- e, e = 2 (D + 8) 2^-24 S +
2^-20 (exponential, rescaling), and enters the product with the values to
2^-16 relative or better, and the fp32 sums over n tokens add at most n 2^-24.
So |out - formula| <= eps/2 |out| + (e + 2^-16 + n 2^-23) sum p |v| (plus the
half step 2^-25 of fp16's subnormals), and |lse - formula| <= e + n 2^-23 +
2^-22 |lse|."""
import math

import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def case(lengths, hq=6, hk=2, D=128, dtype="f16", kv="f16", page=16, window=0, seed=1, spread=1.5, extra=2, width=None,
         stale=0.0):
    """Caches whose unused slots hold `stale` (NaN, inf, anything)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lengths)
    need = [-(-max(n, 0) // page) for n in lengths]
    width = width or max(max(need), 1)
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    caches = [torch.full((pages, hk, page, D), stale).to(TYPES[kv]) for _ in range(2)]
    at = 0
    for b, n in enumerate(lengths):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for i in range(need[b]):
            m = min(page, n - i * page)
            for x in caches:
                x[table[b, i], :, :m] = (torch.randn((hk, m, D), generator=g) * (40.0 if kv == "e4m3" else 1.0)).to(TYPES[kv])
    scales = [torch.rand((hk,), generator=g) * 0.01 + 0.015 if kv == "e4m3" else None for _ in range(2)]
    q = (torch.randn((B, hq * D), generator=g) * spread).to(TYPES[dtype])
    return dict(lengths=list(lengths), hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=page, window=window, pages=pages,
                table=table, caches=caches, scales=scales, q=q, scale=D ** -0.5)


def formula(c):
    """(out, lse, out's tolerance, lse's tolerance) in 64 bits."""
    B, hq, hk, D, page = len(c["lengths"]), c["hq"], c["hk"], c["D"], c["page"]
    out, lse = np.zeros((B, hq, D)), np.full((B, hq), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    q = c["q"].double().numpy().reshape(B, hq, D)
    eps = torch.finfo(TYPES[c["dtype"]]).eps / 2
    for b, n in enumerate(c["lengths"]):
        n = min(n, c["table"].shape[1] * page)
        lo = max(0, n - c["window"]) if c["window"] else 0
        t = np.arange(lo, max(n, lo))
        pg = c["table"][b].numpy()[t // page]
        t, pg = t[(pg >= 0) & (pg < c["pages"])], pg[(pg >= 0) & (pg < c["pages"])]
        if not len(t):
            continue
        for h in range(hq):
            kh = h // (hq // hk)
            k, v = (x[torch.from_numpy(pg).long(), kh, torch.from_numpy(t % page).long()].double().numpy() for x in c["caches"])
            if c["scales"][0] is not None:
                k, v = k * float(c["scales"][0][kh]), v * float(c["scales"][1][kh])
            s = k @ q[b, h] * c["scale"]
            size = (np.abs(k) @ np.abs(q[b, h])).max() * abs(c["scale"])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            lse[b, h] = m + math.log(l)
            out[b, h] = p @ v / l
            e = 2 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -20
            tol[b, h] = eps * np.abs(out[b, h]) + (e + 2.0 ** -16 + len(t) * 2.0 ** -23) * (p @ np.abs(v) / l) + 2.0 ** -25
            ltol[b, h] = e + len(t) * 2.0 ** -23 + 2.0 ** -22 * abs(lse[b, h])
    return out, lse, tol, ltol


class Device:
    def __init__(self, c, workspace=None):
        self.c, dev = c, "cuda"
        self.d = bgg.bgg_cache_describe(c["kv"], c["pages"], c["page"], c["hk"], c["D"])
        self.k, self.v = (x.to(dev) for x in c["caches"])
        self.ks, self.vs = (None if x is None else x.to(dev) for x in c["scales"])
        self.table, self.q = c["table"].to(dev), c["q"].to(dev)
        self.n = torch.tensor(c["lengths"], dtype=torch.int32, device=dev)
        B = len(c["lengths"])
        self.out = torch.full((B, c["hq"] * c["D"]), float("nan"), dtype=TYPES[c["dtype"]], device=dev)
        self.lse = torch.full((B, c["hq"]), float("nan"), device=dev)
        self.ws = workspace if workspace is not None else bgg.workspace(bgg.bgg_attention_workspace_size(self.d, c["hq"], B))

    def step(self, stream=None):
        bgg.bgg_paged_attention(self.d, self.k, self.v, self.table, self.n, self.q, self.out, self.ws,
                                scale=self.c["scale"], window=self.c["window"], lse=self.lse, k_scale=self.ks,
                                v_scale=self.vs, stream=stream)

    def check(self):
        c = self.c
        torch.cuda.synchronize()
        out, lse, tol, ltol = formula(c)
        got = self.out.double().cpu().numpy().reshape(out.shape)
        gl = self.lse.double().cpu().numpy()
        bad = ~(np.abs(got - out) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], out[bad][:5], tol[bad][:5])
        empty = np.isinf(lse)
        assert np.array_equal(gl == -np.inf, empty)
        off = np.abs(gl[~empty] - lse[~empty])
        assert np.all(off <= ltol[~empty]), (off.max(), ltol.min())


def run_check(c):
    d = Device(c)
    d.step()
    d.check()
    assert not d.ws[:16384].any(), "the counters are zero again"
    return d


@pytest.mark.parametrize("dtype,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hk", [(6, 1), (4, 4), (32, 2)])
def test_every_type_and_head(dtype, kv, D, hq, hk):
    run_check(case([1, 37, 300, 0, 16], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=32, seed=D))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1023, 2049])
@pytest.mark.parametrize("page", [16, 64])
def test_lengths(n, page):
    run_check(case([n], hq=12, hk=2, page=page, seed=n))


@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (16, 1), (17, 1), (33, 1), (40, 2), (48, 8), (24, 4), (64, 64)])
def test_head_groups(hq, hk):
    run_check(case([90, 7], hq=hq, hk=hk, D=64, dtype="bf16", kv="bf16"))


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
def test_page_sizes(page):
    run_check(case([1000, 3, page, page + 1, max(page - 1, 1)], page=page, kv="e4m3"))


@pytest.mark.parametrize("window", [1, 2, 16, 31, 33, 100, 5000])
def test_windows(window):
    run_check(case([1, 40, 99, 333, 0], window=window, hq=8, hk=4, D=64))


def test_ragged_batch():
    rng = np.random.default_rng(5)
    lengths = [int(v) for v in np.exp(rng.uniform(0, math.log(3000), 37))] + [0, 6000]
    run_check(case(lengths, hq=12, hk=4, D=128, dtype="bf16", kv="bf16", page=64))


def test_large_batch_with_a_few_long_sequences():
    """More than 64 sequences (several per lane of the schedule), some cut in
    chunks."""
    lengths = [1 + (i * 13) % 40 for i in range(150)]
    for b in (0, 63, 64, 149):
        lengths[b] = 3000 + b
    lengths[77] = 0
    run_check(case(lengths, hq=8, hk=1, D=64, page=32, seed=31))


def test_largest_batch():
    lengths = [(i * 7) % 4 for i in range(4096)]
    lengths[2048], lengths[4095] = 900, 700
    run_check(case(lengths, hq=2, hk=1, D=64, kv="e4m3", seed=32))


@pytest.mark.parametrize("hq,hk", [(4096, 1), (1024, 1024), (4096, 512)])
def test_largest_head_counts(hq, hk):
    run_check(case([40, 3], hq=hq, hk=hk, D=64, seed=33))


def test_largest_page_and_one_wide_table():
    run_check(case([70000, 5], hq=2, hk=1, D=64, page=65536, seed=34))
    run_check(case([40], hq=2, hk=1, D=64, page=16, width=(1 << 31) // 16 - 1, seed=34))


def test_subnormal_keys_and_values_count():
    """fp16 values below 2^-14 are not flushed."""
    c = case([300], hq=4, hk=1, D=64, seed=35)
    for x in c["caches"]:
        x *= 2.0 ** -22
    c["scale"] = 2.0 ** 20
    assert (c["caches"][0].abs() < 2.0 ** -14).all() and c["caches"][0].any()
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    out, lse, tol, ltol = formula(c)
    got = d.out.double().cpu().numpy().reshape(out.shape)
    assert np.all(np.abs(got - out) <= tol) and np.abs(got).max() > 2.0 ** -24
    assert np.all(np.abs(d.lse.double().cpu().numpy() - lse) <= ltol)


def test_two_streams_with_their_own_workspaces():
    """Calls that overlap in time."""
    cs = [case([5000, 40], hq=12, hk=2, seed=41), case([3000] * 3, hq=8, hk=4, D=64, seed=42)]
    ds = [Device(c) for c in cs]
    for d in ds:
        d.step()
    torch.cuda.synchronize()
    want = [d.out.clone() for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    for d in ds:
        d.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(ds, streams):
            d.step(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(d.out, w) for d, w in zip(ds, want))


def test_many_short_sequences():
    run_check(case([1 + (i * 7) % 50 for i in range(300)], hq=4, hk=2, D=64))


def test_lengths_past_the_table_and_below_zero():
    c = case([40, 64], page=16)
    c["lengths"] = [-5, 1 << 30]
    run_check(c)


@pytest.mark.parametrize("stale", [float("nan"), float("inf"), -65504.0])
@pytest.mark.parametrize("kv", ["f16", "e4m3"])
@pytest.mark.parametrize("window", [0, 21])
def test_hidden_tokens_have_no_influence(stale, kv, window):
    """Slots past a length, pages of other sequences and tokens before the
    window hold NaN, inf or large values."""
    lengths = [1, 17, 50, 95, 0]
    clean = case(lengths, page=32, kv=kv, window=window, seed=4)
    dirty = case(lengths, page=32, kv=kv, window=window, seed=4, stale=stale)
    if window:
        for c in (dirty,):
            for b, n in enumerate(lengths):
                for t in range(max(0, n - window)):
                    for x in c["caches"]:
                        x[c["table"][b, t // 32], :, t % 32] = torch.tensor(stale).to(TYPES[kv])
    a, b = run_check(clean), Device(dirty)
    b.step()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_pages_outside_the_cache_hide_their_tokens():
    c = case([200, 60, 33], page=16, seed=6)
    c["table"][0, 3], c["table"][0, 7], c["table"][1, :] = -1, c["pages"], -7
    c["table"][2, 2] = 2 ** 31 - 1
    run_check(c)


def test_large_and_equal_scores():
    c = case([70, 300], spread=60.0, seed=9)  # softmax of a few tokens
    run_check(c)
    c = case([70, 300], seed=9)
    c["caches"][0][:] = 0.25  # every score the same
    run_check(c)
    c["scale"] = 0.0
    run_check(c)
    c = case([70, 300], seed=10)
    c["scale"] = -0.7
    run_check(c)


def test_scores_of_minus_infinity():
    c = case([40, 50], hq=2, hk=1, D=64, seed=12)
    c["q"][:] = 1.0
    c["caches"][0][c["table"][0, 0], :, 3] = float("-inf")  # one token of sequence 0 never counts
    for i in range(4):  # no token of sequence 1 counts
        c["caches"][0][c["table"][1, i]] = float("-inf")
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    assert not d.out[1].any() and torch.all(d.lse[1] == -math.inf)
    keep = [t for t in range(40) if t != 3]
    k, v = (x[c["table"][0, torch.tensor(keep) // 16].long(), 0, torch.tensor(keep) % 16].double() for x in c["caches"])
    s = k.sum(-1) * c["scale"]
    p = torch.softmax(s, 0)
    # (sums as in the module's note, with S of this row)
    tol = 2.0 ** -11 * (p @ v).abs() + (2 * 72 * 2.0 ** -24 * float(k.abs().sum(-1).max()) * c["scale"] + 2.0 ** -15) * (p @ v.abs())
    assert torch.all((d.out[0, :64].double().cpu() - p @ v).abs() <= tol)


def test_nan_of_a_visible_token_shows():
    c = case([40, 50], hq=2, hk=1, D=64, seed=12)
    c["caches"][0][c["table"][0, 1], :, 3, 5] = float("nan")
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    assert torch.isnan(d.out[0]).all() and torch.isnan(d.lse[0]).all()
    assert torch.isfinite(d.out[1]).all()


def test_same_bits_again_and_in_another_batch():
    """A sequence's result depends neither on the run nor on the pages that
    hold it."""
    c = case([3000, 700, 12], hq=12, hk=2, page=64, seed=3)
    a = run_check(c)
    first = a.out.clone()
    for _ in range(5):
        a.step()
        torch.cuda.synchronize()
        assert torch.equal(a.out, first)
    perm = torch.randperm(c["pages"])
    moved = dict(c, caches=[x[perm] for x in c["caches"]], table=torch.argsort(perm)[c["table"].clamp(min=0).long()].int())
    b = Device(moved)
    b.step()
    torch.cuda.synchronize()
    assert torch.equal(b.out, first)


def test_rows_of_a_wider_buffer_and_table():
    c = case([100, 45], hq=8, hk=4, D=96, dtype="bf16", kv="bf16", seed=21)
    d = Device(c)
    n = 8 * 96
    wide = torch.full((2, 3 * n), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, n:2 * n] = d.q
    big = torch.full((2, c["table"].shape[1] + 9), 5, dtype=torch.int32, device="cuda")
    big[:, :c["table"].shape[1]] = d.table
    d.table = big[:, :c["table"].shape[1]]
    d.q, d.out = wide[:, n:2 * n], wide[:, 2 * n:]
    d.step()
    d.check()
    assert torch.all(wide[:, :n] == 7.0)


def test_offsets_past_32_bits():
    """Pages whose value offsets pass 2^31 and byte offsets 2^32."""
    hk, page, D = 8, 64, 256
    pages = (1 << 31) // (hk * page * D) + 8
    c = case([100, 130], hq=8, hk=hk, D=D, page=page, seed=2)
    small = c["caches"]
    where = torch.tensor([pages - 1, pages - 3, 0, pages - 6, 2, pages - 2, 1])[:c["pages"]]
    d = Device(dict(c, caches=[x[:1] for x in small]))
    d.d = bgg.bgg_cache_describe("f16", pages, page, hk, D)
    d.k = torch.empty((pages, hk, page, D), dtype=torch.float16, device="cuda")
    d.v = torch.empty_like(d.k)
    for i, w in enumerate(where.tolist()):
        d.k[w], d.v[w] = small[0][i].cuda(), small[1][i].cuda()
    d.table = torch.where(c["table"] >= 0, where[c["table"].clamp(min=0).long()].int(), c["table"]).cuda()
    d.ws = bgg.workspace(bgg.bgg_attention_workspace_size(d.d, 8, 2))
    d.c = c
    d.step()
    d.check()


def test_long_context_sampled():
    """One sequence of 70001 tokens on one key head."""
    run_check(case([70001], hq=4, hk=1, D=128, page=256, seed=13))


def test_one_workspace_for_calls_of_every_size():
    """Calls in stream order share a workspace; also two captured graphs,
    replayed in turn with eager calls between them."""
    cs = [case([900, 30], hq=12, hk=2, seed=1), case([5] * 9, hq=4, hk=4, D=64, seed=2), case([2500], hq=32, hk=2, seed=3),
          case([10] * 30 + [300 + 90 * i for i in range(12)], hq=16, hk=16, D=64, seed=4)]
    ds = [Device(c) for c in cs]
    ws = bgg.workspace(max(d.ws.numel() for d in ds))
    want = []
    for d in ds:
        d.step()
        torch.cuda.synchronize()
        want.append((d.out.clone(), d.lse.clone()))
        d.ws = ws
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for d in ds[:2]:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                d.step()
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for d in ds:
            d.out.zero_()
            d.lse.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        ds[2].step()
        graphs[1].replay()
        ds[3].step()
        torch.cuda.synchronize()
        for d, (o, l) in zip(ds, want):
            assert torch.equal(d.out, o) and torch.equal(d.lse, l)
    assert not ws[:16384].any()


def test_lengths_that_grow_between_replays():
    """A captured step reads lengths and page table when it runs."""
    c = case([400, 33], seed=17)
    d = Device(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        d.step()
    torch.cuda.synchronize()
    for lengths in ([1, 0], [399, 20], [400, 33], [200, 1]):
        d.n.copy_(torch.tensor(lengths, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        d.c = dict(c, lengths=lengths)
        d.check()


def test_a_used_workspace_is_reset():
    c = case([2000], seed=1)
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    want = d.out.clone()
    d.ws.fill_(255)
    n = d.ws.numel() // 16 * 16
    bgg.bgg_gemv_workspace_reset(d.ws[:n])
    d.step()
    torch.cuda.synchronize()
    assert torch.equal(d.out, want)


def test_without_lse():
    d = Device(case([77], seed=2))
    d.lse = None
    d.step()
    torch.cuda.synchronize()
    out, _, tol, _ = formula(d.c)
    assert np.all(np.abs(d.out.double().cpu().numpy().reshape(out.shape) - out) <= tol)


def test_binding_refusals():
    d = Device(case([20, 30], seed=2))
    good = (d.d, d.k, d.v, d.table, d.n, d.q, d.out, d.ws)

    def call(i, x, **kw):
        a = list(good)
        a[i] = x
        bgg.bgg_paged_attention(*a, **dict(dict(scale=0.1), **kw))

    for i, x in ((1, d.k[1:]), (2, d.v.float()), (3, d.table[:1]), (3, d.table.long()), (3, d.table.t()), (4, d.n[:1]),
                 (4, d.n.long()), (5, d.q.float()), (5, d.q[:, :-1]), (6, d.out[:, :128]), (6, d.out.cpu()), (5, d.q.cpu()),
                 (7, d.ws.cpu())):
        with pytest.raises(ValueError):
            call(i, x)
    for i, x, kw in ((7, d.ws[:64], {}), (0, d.d, dict(window=-1)), (0, d.d, dict(scale=math.nan))):
        with pytest.raises(bgg.BggError):
            call(i, x, **kw)
    bgg.bgg_paged_attention(d.d, d.k, d.v, d.table[:0], d.n[:0], d.q[:0], d.out[:0], d.ws, scale=0.1)
    torch.cuda.synchronize()


def test_unfilled_descriptors_are_refused():
    """A descriptor that bgg_cache_describe never filled (a head dimension of
    zero), or one changed afterwards, is an error."""
    d = Device(case([20, 30], seed=2))
    T = len(d.q)
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    freqs = torch.ones(d.d.head_dim // 2, device="cuda")
    changed = bgg.bgg_cache_desc.from_buffer_copy(d.d)
    changed.page_size *= 2
    for c, error in ((bgg.bgg_cache_desc(), ValueError), (changed, bgg.BggError)):
        with pytest.raises(error):
            bgg.bgg_paged_attention(c, d.k, d.v, d.table, d.n, d.q, d.out, d.ws, scale=0.1)
        with pytest.raises(error):
            bgg.bgg_rotary_append(c, None, None, pos, slots, freqs, q=d.q, q_out=torch.empty_like(d.q))
    torch.cuda.synchronize()
