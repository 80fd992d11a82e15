"""Attention of groups of sequences that share their first pages against the
formula in 64 bits.

Tolerances.  Those of test_gpu_attention (scores, statistics, sums), and the
rounding of the shared part's probabilities to one 16-bit term: half a step u
of it (eps/2 of the values' type, fp16 for an E4M3 cache), at most
u sum p |v| / sum p over the tokens.  Below fp16's normal range, 2^-14 after
the lift of 2^7, the half step is 2^-25, so a probability below 2^-21 of its
row's maximum is off by up to 2^-32 of the maximum: 2^-32 sum |v| / sum p
more, with sum p >= 1."""
import math

import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg
from test_gpu_attention import TYPES

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def case(groups, hq=6, hk=2, D=128, dtype="f16", kv="f16", page=16, window=0, seed=1, spread=1.5, outside=(), stale=0.0,
         own_entries=True):
    """groups: [(pages shared, [tokens of each member beyond them; below 0:
    shorter than the prefix; None: an unused slot])]; outside: lengths of
    sequences of no group, before the first.  Cells that no token uses hold
    `stale`."""
    g = torch.Generator().manual_seed(seed)
    lengths, starts, shared = list(outside), [len(outside)], [0] * len(outside)
    for pages, own in groups:
        lengths += [0 if n is None else max(0, pages * page + n) for n in own]
        shared += [pages] * len(own)
        starts.append(len(lengths))
    B = len(lengths)
    mine = [max(0, -(-n // page) - s) for n, s in zip(lengths, shared)]
    width = max(1, max(s + m for s, m in zip(shared, mine)) if B else 1)
    total = sum(mine) + sum(p for p, _ in groups) + 2
    order = torch.randperm(total, generator=g).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    full = table.clone()  # as a call without groups would have it
    caches = [torch.full((total, hk, page, D), stale).to(TYPES[kv]) for _ in range(2)]

    def write(p, m):
        for x in caches:
            x[p, :, :m] = (torch.randn((hk, m, D), generator=g) * (40.0 if kv == "e4m3" else 1.0)).to(TYPES[kv])

    at = 0
    for (pages, own), s in zip(groups, starts):
        pre = order[at:at + pages]
        at += pages
        for p in pre:
            write(int(p), page)
        for b in range(s, s + len(own)):
            full[b, :pages] = pre
            if b == s or own_entries:
                table[b, :pages] = pre
    for b in range(B):
        for i in range(mine[b]):
            p = int(order[at])
            at += 1
            table[b, shared[b] + i] = full[b, shared[b] + i] = p
            write(p, min(page, lengths[b] - (shared[b] + i) * page))
    scales = [torch.rand((hk,), generator=g) * 0.01 + 0.015 if kv == "e4m3" else None for _ in range(2)]
    q = (torch.randn((B, hq * D), generator=g) * spread).to(TYPES[dtype])
    return dict(lengths=lengths, hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=page, window=window, pages=total, table=table,
                full=full, caches=caches, scales=scales, q=q, scale=D ** -0.5, starts=starts, shared=shared)


def formula(c, rows=None):
    """{(sequence, head): (out, lse, out's tolerance, lse's)} in 64 bits."""
    B, hq, hk, D, page = len(c["lengths"]), c["hq"], c["hk"], c["D"], c["page"]
    q = c["q"].double().numpy().reshape(B, hq, D)
    eps = torch.finfo(TYPES[c["dtype"]]).eps / 2
    u = torch.finfo(TYPES["f16" if c["kv"] == "e4m3" else c["kv"]]).eps / 2
    got, kept = {}, {}
    for b, h in rows if rows is not None else [(b, h) for b in range(B) for h in range(hq)]:
        n = min(max(c["lengths"][b], 0), c["full"].shape[1] * page)
        lo = max(0, n - c["window"]) if c["window"] else 0
        kh = h // (hq // hk)
        if (b, kh) not in kept:
            t = np.arange(lo, max(n, lo))
            pg = c["full"][b].numpy()[t // page]
            ok = (pg >= 0) & (pg < c["pages"])
            t, pg = torch.from_numpy(t[ok] % page).long(), torch.from_numpy(pg[ok]).long()
            k, v = (x[pg, kh, t].double().numpy() for x in c["caches"])
            if c["scales"][0] is not None:
                k, v = k * float(c["scales"][0][kh]), v * float(c["scales"][1][kh])
            kept = {(b, kh): (k, v)}
        k, v = kept[b, kh]
        if not len(k):
            got[b, h] = np.zeros(D), -np.inf, np.zeros(D), 0.0
            continue
        s = k @ q[b, h] * c["scale"]
        size = (np.abs(k) @ np.abs(q[b, h])).max() * abs(c["scale"])
        m = s.max()
        p = np.exp(s - m)
        l = p.sum()
        o, x = p @ v / l, m + math.log(l)
        e = 2 * (D + 8) * 2.0 ** -24 * size + 2.0 ** -20
        tol = eps * np.abs(o) + (e + 2.0 ** -16 + u + len(k) * 2.0 ** -23) * (p @ np.abs(v) / l) + 2.0 ** -25
        tol = tol + 2.0 ** -32 * np.abs(v).sum(0) / l
        got[b, h] = o, x, tol, e + len(k) * 2.0 ** -23 + 2.0 ** -22 * abs(x)
    return got


class Device:
    def __init__(self, c, workspace=None):
        self.c, dev = c, "cuda"
        self.d = bgg.bgg_cache_describe(c["kv"], c["pages"], c["page"], c["hk"], c["D"])
        self.k, self.v = (x.to(dev) for x in c["caches"])
        self.ks, self.vs = (None if x is None else x.to(dev) for x in c["scales"])
        self.table, self.q = c["table"].to(dev), c["q"].to(dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.n, self.starts = torch.tensor(c["lengths"], **i32), torch.tensor(c["starts"], **i32)
        self.shared = torch.tensor(c["shared"], **i32)
        B = len(c["lengths"])
        self.out = torch.full((B, c["hq"] * c["D"]), NAN, dtype=TYPES[c["dtype"]], device=dev)
        self.lse = torch.full((B, c["hq"]), NAN, device=dev)
        size = bgg.bgg_shared_attention_workspace_size(self.d, c["hq"], B)
        self.ws = workspace if workspace is not None else bgg.workspace(size)

    def step(self, stream=None):
        c = self.c
        bgg.bgg_shared_attention(self.d, self.k, self.v, self.table, self.n, self.starts, self.shared, self.q, self.out,
                                 self.ws, scale=c["scale"], window=c["window"], lse=self.lse, k_scale=self.ks,
                                 v_scale=self.vs, stream=stream)

    def check(self, rows=None):
        torch.cuda.synchronize()
        B, hq, D = len(self.c["lengths"]), self.c["hq"], self.c["D"]
        out, lse = self.out.double().cpu().numpy().reshape(B, hq, D), self.lse.double().cpu().numpy()
        for (b, h), (o, x, tol, ltol) in formula(self.c, rows).items():
            bad = ~(np.abs(out[b, h] - o) <= tol)
            assert not bad.any(), (b, h, np.argwhere(bad)[:5].ravel(), out[b, h][bad][:5], o[bad][:5], tol[bad][:5])
            assert (lse[b, h] == -np.inf) == (x == -np.inf), (b, h, lse[b, h], x)
            assert x == -np.inf or abs(lse[b, h] - x) <= ltol, (b, h, lse[b, h], x, ltol)


def run_check(c, rows=None):
    d = Device(c)
    d.step()
    d.check(rows)
    assert not d.ws[:16384].any(), "the counters are zero again"
    return d


@pytest.mark.parametrize("dtype,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hk", [(6, 1), (4, 4), (32, 2)])
def test_every_type_and_head(dtype, kv, D, hq, hk):
    run_check(case([(3, [1, 37, 300, None, 16]), (2, [5])], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=32, seed=D))


@pytest.mark.parametrize("pages", [1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 32, 33, 63, 65])
@pytest.mark.parametrize("page", [16, 64])
def test_prefix_lengths(pages, page):
    """Prefixes that end inside a tile of 32 tokens among them."""
    run_check(case([(pages, [1, 20, 0])], hq=12, hk=2, page=page, seed=pages))


@pytest.mark.parametrize("own", [[0, 0, 0], [1, 1], [-1, 5, -16], [-40, -47, -48, -1000, 3], [None, None], [None, 7], [600, 1, 2000]])
def test_own_tokens(own):
    """None beyond the prefix, fewer tokens than the prefix, several chunks."""
    run_check(case([(3, own)], hq=8, hk=2, D=64, seed=len(own)))


@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (16, 1), (17, 1), (33, 1), (40, 2), (48, 8), (24, 4), (64, 64)])
@pytest.mark.parametrize("members", [1, 2, 9, 40])
def test_rows_of_a_group(hq, hk, members):
    """From one row to several row blocks, with a last one of any size."""
    run_check(case([(4, [1 + (7 * i) % 40 for i in range(members)])], hq=hq, hk=hk, D=64, dtype="bf16", kv="bf16", seed=hq))


@pytest.mark.parametrize("window", [1, 2, 31, 48, 49, 50, 64, 65, 100, 5000])
def test_windows(window):
    run_check(case([(3, [1, 40, 99, 17, None, -20]), (9, [3, 60])], window=window, hq=8, hk=4, D=64, outside=[33, 0, 1]))


def test_groups_of_every_kind():
    run_check(case([(1, [3]), (0, [5, 40]), (6, [1] * 17), (2, []), (2, [None]), (30, [9, 100]), (0, [])], hq=6, hk=3, D=96,
                   dtype="bf16", kv="e4m3", outside=[1, 200, 0], seed=3))


def test_sequences_behind_the_last_group():
    c = case([(4, [3, 9]), (0, [50, 700])], hq=4, hk=2, D=64)
    c["starts"] = c["starts"][:2]  # the last two belong to no group
    run_check(c)


def test_no_groups_is_paged_attention():
    c = case([(4, [3, 9, 600])], hq=4, hk=2, D=64)
    c["starts"] = [0]
    d = run_check(c)
    out = torch.empty_like(d.out)
    bgg.bgg_paged_attention(d.d, d.k, d.v, d.table, d.n, d.q, out, d.ws, scale=c["scale"])
    assert torch.equal(out, d.out)


def test_only_the_first_member_names_the_shared_pages():
    """The others' entries there are not read, nor their counts."""
    c = case([(5, [3, 9, 600]), (2, [1, 30])], hq=4, hk=2, D=64, own_entries=False)
    c["shared"][1], c["shared"][2], c["shared"][4] = 0, 99, -5
    run_check(c)


def test_one_group_per_sequence_and_large_batches():
    run_check(case([((7 * i) % 5, [1 + i % 33]) for i in range(150)], hq=4, hk=2, D=64, seed=5))
    run_check(case([(3, [(i * 5) % 23 for i in range(300)]), (70, [2] * 70)], hq=4, hk=1, D=64, kv="e4m3", seed=6),
              rows=[(b, h) for b in range(0, 370, 7) for h in (0, 3)])


def test_largest_batch():
    c = case([(2, [i % 5 for i in range(2000)])] + [(1, [i % 3]) for i in range(96)] + [(40, [1] * 2000)], hq=2, hk=1, D=64,
             kv="e4m3", seed=8)
    run_check(c, rows=[(b, b % 2) for b in list(range(0, 4096, 37)) + list(range(1990, 2110)) + [4095]])


@pytest.mark.parametrize("D,hq,hk", [(64, 48, 8), (128, 12, 2), (256, 4, 1)])
def test_long_prefixes_in_several_chunks(D, hq, hk):
    c = case([(130, [1, 70, 40, None, 900] * 3), (3, [4])], hq=hq, hk=hk, D=D, page=64, dtype="bf16", kv="bf16", seed=D)
    run_check(c, rows=[(b, h) for b in range(16) for h in (0, hq // 2, hq - 1)])


def test_many_tiles_per_wave():
    """So many rows that a workgroup takes the whole prefix: more than 64
    tiles for a wave, whose page numbers are loaded 64 at a time."""
    c = case([(565, [1, 3, 0, 17, 2, 1, 5, 40])], hq=4096, hk=8, D=64, seed=9)
    run_check(c, rows=[(b, h) for b in (0, 3, 7) for h in (0, 511, 512, 2000, 4095)])


def test_largest_page():
    run_check(case([(1, [5, 70])], hq=2, hk=1, D=64, page=65536, seed=34))


def test_pages_that_a_window_left():
    """Entries of the first member outside the cache hide their tokens from
    the whole group."""
    c = case([(6, [3, 9, 20])], hq=4, hk=2, D=64, stale=NAN)
    for e, v in ((1, -1), (2, c["pages"]), (5, -(1 << 31))):
        c["table"][0, e] = v
        c["full"][:, e] = -1
    run_check(c)
    c = case([(3, [3, 9])], hq=4, hk=2, D=64)
    c["table"][0, :3], c["full"][:, :3] = -1, -1
    run_check(c)


@pytest.mark.parametrize("starts", [[0, 3, 1, 5], [-7, 2, 99, 5], [5, 5, 0, 0], [9, 9, 9, 9], [3, 2, 1, 0], [0, 5, 0, 5]])
def test_starts_that_do_not_rise(starts):
    """Cut to 0 .. B, and none below an earlier one."""
    c = case([(4, [3, 9, 20, 0, 55])], hq=4, hk=2, D=64, own_entries=True)
    c["starts"] = starts
    run_check(c)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 96, 256])
@pytest.mark.parametrize("window", [0, 50])
def test_what_hidden_tokens_hold_has_no_influence(kv, D, window):
    """Keys and values that some members of a group see and others do not
    (shorter sequences, windows), NaN and infinite there: the others' results
    are those of a clean cache, bit for bit."""
    c = case([(7, [20, -30, -1, None, -100, 5])], hq=6, hk=2, D=D, dtype="bf16" if kv == "bf16" else "f16", kv=kv, window=window,
             seed=D)
    clean = Device(c)
    clean.step()
    bad = Device(c)
    page, table = c["page"], c["full"][0].tolist()
    seen = [(max(0, n - window) if window else 0, n) for n in c["lengths"]]
    for t in (95, 110, 111, 85, 3):
        for x in (bad.k, bad.v):
            x[table[t // page], :, t % page, 1] = NAN
            if kv != "e4m3":
                x[table[t // page], :, t % page, 2] = -INF
    bad.step()
    torch.cuda.synchronize()
    for b, (lo, n) in enumerate(seen):
        if not any(lo <= t < n for t in (95, 110, 111, 85, 3)):
            assert torch.equal(clean.out[b], bad.out[b]) and torch.equal(clean.lse[b], bad.lse[b]), b
        else:
            assert torch.isnan(bad.out[b]).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,hq,hk", [(64, 2, 1), (96, 6, 2), (128, 12, 1), (192, 3, 3), (256, 16, 1)])
@pytest.mark.parametrize("window", [0, 130])
def test_infinite_values(dtype, D, hq, hk, window):
    """An infinite value of a visible token makes its element infinite, NaN
    where both signs or a NaN meet; rows that do not see it and other
    elements are as without.  Prefix of 160 tokens, one member shorter."""
    c = case([(10, [1, 30, -60, 700])], hq=hq, hk=hk, D=D, dtype=dtype, kv=dtype, window=window, seed=D)
    c["q"] = c["q"].abs() + 0.5
    page = c["page"]
    planted = [(5, {3: INF}), (6, {159: -INF}), (7, {0: INF, 130: INF}), (8, {100: INF, 120: -INF}), (9, {99: INF, 125: NAN}),
               (10, {140: -INF}), (D - 1, {100: INF}), (D - 2, {158: INF, 20: -INF})]
    caches = [x.clone() for x in c["caches"]]
    k = caches[0]
    k[int(c["full"][0, 140 // page]), :, 140 % page] = -300.0  # a probability of zero
    c["caches"] = caches
    clean = dict(c, caches=[x.clone() for x in caches])
    for dim, tokens in planted:
        for t, v in tokens.items():
            caches[1][int(c["full"][0, t // page]), :, t % page, dim] = v
            clean["caches"][1][int(c["full"][0, t // page]), :, t % page, dim] = 0.0
    got, want = Device(c), Device(clean)
    got.step(), want.step()
    torch.cuda.synchronize()
    B = len(c["lengths"])
    out, ref = got.out.view(B, hq, D), want.out.view(B, hq, D).clone()
    for b, n in enumerate(c["lengths"]):
        lo = max(0, n - window) if window else 0
        for dim, tokens in planted:
            v = sum(x for t, x in tokens.items() if lo <= t < n)
            if v != 0:
                ref[b, :, dim] = v
    assert torch.equal(got.lse, want.lse)
    same = (out == ref) | (torch.isnan(out) & torch.isnan(ref))
    assert same.all(), (~same).nonzero()[:8]


def test_scores_of_minus_infinity():
    """A row whose every score is -inf gives 0 and -inf, whatever its values;
    one with -inf in the prefix alone has its own tokens' result."""
    c = case([(4, [0, 25])], hq=2, hk=1, D=64)
    c["q"] = c["q"].abs() + 0.5
    for e in range(4):
        c["caches"][0][int(c["full"][0, e])] = -INF
        c["caches"][1][int(c["full"][0, e])] = NAN
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    assert (d.out[0] == 0).all() and (d.lse[0] == -INF).all()
    assert torch.isfinite(d.lse[1]).all()
    # (its lse is that of its own tokens; a NaN value of a visible token makes its elements NaN)
    assert torch.isnan(d.out[1]).all()
    own = case([(0, [25])], hq=2, hk=1, D=64)
    own["caches"] = c["caches"]
    own["pages"], own["table"], own["full"] = c["pages"], c["full"][1:, 4:], c["full"][1:, 4:]
    own["q"] = c["q"][1:]
    x = formula(own)
    assert all(abs(d.lse[1, h].item() - x[0, h][1]) <= x[0, h][3] for h in range(2))


def test_nan_and_infinite_queries_stay_in_their_rows():
    c = case([(5, [3, 9, 20])], hq=4, hk=2, D=64)
    clean = Device(c)
    clean.step()
    bad = Device(c)
    bad.q[1, 5] = NAN
    bad.q[1, 64 + 5] = INF
    bad.step()
    torch.cuda.synchronize()
    for b in (0, 2):
        assert torch.equal(clean.out[b], bad.out[b]) and torch.equal(clean.lse[b], bad.lse[b])
    assert torch.isnan(bad.out[1, :128]).all() and torch.equal(bad.out[1, 128:], clean.out[1, 128:])


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
def test_scales(scale):
    c = case([(5, [3, -9, 20])], hq=4, hk=2, D=64, spread=1.0)
    c["scale"] = scale
    run_check(c)


def test_large_values_of_bfloat16():
    """Values near the top of the range do not overflow the sums."""
    c = case([(40, [3, 20])], hq=4, hk=1, D=64, dtype="bf16", kv="bf16")
    c["caches"][1] = torch.full_like(c["caches"][1], 3e38)
    d = Device(c)
    d.step()
    torch.cuda.synchronize()
    want = torch.tensor(3e38).bfloat16().float().item()
    assert ((d.out.float() - want).abs() <= 2.0 ** -7 * want).all()


def test_strides_and_output_in_the_place_of_the_queries():
    c = case([(5, [3, 9, 20]), (1, [4])], hq=4, hk=2, D=64)
    d = Device(c)
    want = Device(c)
    want.step()
    wide = torch.full((4, 4 * 64 + 24), 7.0, dtype=torch.float16, device="cuda")
    wide[:, 8:8 + 256] = d.q
    d.q = d.out = wide[:, 8:8 + 256]
    table = torch.full((4, d.table.shape[1] + 3), 5, dtype=torch.int32, device="cuda")
    table[:, :-3] = d.table
    d.table = table[:, :-3]
    d.step()
    torch.cuda.synchronize()
    assert torch.equal(d.out, want.out)
    assert (wide[:, :8] == 7).all() and (wide[:, 264:] == 7).all()


def test_one_workspace_for_both_attentions_and_two_streams():
    """A workspace passes between calls of different shapes; calls that
    overlap in time have their own."""
    big = case([(40, [1, 900, 30]), (3, [700])], hq=12, hk=2, page=64, seed=1)
    small = case([(2, [5, 6])], hq=4, hk=2, D=64, seed=2)
    ws = bgg.workspace(max(Device(c).ws.numel() for c in (big, small)))
    ds = [Device(c, ws) for c in (big, small)]
    for _ in range(3):
        for d in ds:
            d.out.fill_(NAN)
            d.step()
            out = torch.empty_like(d.out)
            bgg.bgg_paged_attention(d.d, d.k, d.v, d.c["full"].cuda(), d.n, d.q, out, ws, scale=d.c["scale"])
            d.check()
            assert torch.allclose(out.float(), d.out.float(), rtol=2e-3, atol=2e-3)
    pair = [Device(big), Device(small)]
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(pair, streams):
            d.step(stream=s)
    for d in pair:
        d.check()


def test_two_captured_calls_of_one_workspace():
    """Replayed in turn, of different shapes, with eager calls in between."""
    cs = [case([(40, [1, 900, 30]), (3, [700])], hq=12, hk=2, page=64, seed=1), case([(2, [5, 6])], hq=4, hk=2, D=64, seed=2)]
    ws = bgg.workspace(max(Device(c).ws.numel() for c in cs))
    ds, graphs, side = [Device(c, ws) for c in cs], [], torch.cuda.Stream()
    for d in ds:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            d.step()
        graphs.append(graph)
    for i in (0, 1, 1, 0, 0, 1):
        for d in ds:
            d.out.fill_(NAN)
        ds[1 - i].step()
        graphs[i].replay()
        for d in ds:
            d.check()
    assert not ws[:16384].any()


@pytest.mark.parametrize("dtype,kv,D,hq,hk", [("f16", "f16", 128, 8, 2), ("bf16", "bf16", 256, 4, 4), ("f16", "e4m3", 64, 32, 1),
                                              ("bf16", "e4m3", 96, 20, 2)])
def test_large_batches_with_own_tokens_of_every_length(dtype, kv, D, hq, hk):
    """So many sequences and head blocks that one wave takes an item, among
    them sequences long enough to be cut."""
    B = -(-1024 // (hk * -(-hq // hk // 16))) + 1
    own = [(7 * b) % 45 for b in range(B)]
    own[3], own[B // 2], own[B - 1] = 2900, 9000, None
    c = case([(4, own[:B // 3]), (9, own[B // 3:])], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=32, seed=D)
    run_check(c, [(b, h) for b in (0, 3, 4, B // 3 - 1, B // 3, B // 2, B - 2, B - 1) for h in range(hq)])


def test_same_call_same_bits():
    c = case([(130, [1, 70, 40, 900]), (3, [4])], hq=12, hk=2, page=64, dtype="bf16", kv="bf16")
    d = Device(c)
    d.step()
    first = d.out.clone(), d.lse.clone()
    for _ in range(5):
        d.out.fill_(NAN)
        d.step()
        torch.cuda.synchronize()
        assert torch.equal(first[0], d.out) and torch.equal(first[1], d.lse)


def test_captured_call_with_changing_groups():
    c = case([(20, [1, 70, 40]), (5, [200, 4])], hq=8, hk=2, D=64, page=16)
    d = Device(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        d.step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            d.step()
    torch.cuda.synchronize()
    for lengths, starts, shared in (([321, 390, 360, 280, 84], [0, 3, 5], [20, 20, 20, 5, 5]),
                                    ([321, 390, 100, 0, 84], [0, 2, 2], [20, 20, 0, 5, 5]),
                                    ([5, 390, 360, 280, 84], [1, 3, 5], [0, 7, 0, 2, 0]),
                                    ([321, 390, 360, 280, 84], [0, 3, 5], [20, 20, 20, 5, 5])):
        c["lengths"], c["starts"], c["shared"] = lengths, starts, shared
        for x, v in ((d.n, lengths), (d.starts, starts), (d.shared, shared)):
            x.copy_(torch.tensor(v, dtype=torch.int32))
        d.out.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        d.check()
    assert not d.ws[:16384].any()


def test_offsets_past_32_bits():
    """A cache of more than 4 GB whose shared pages lie at its end."""
    page, hk, D, pages = 1024, 4, 256, 1200  # 2 MB a page
    c = case([(2, [5, 3])], hq=8, hk=hk, D=D, page=page, kv="e4m3")
    small = c["pages"]
    caches = [torch.zeros((pages * 2, hk, page, D), dtype=torch.uint8, device="cuda").view(TYPES["e4m3"]) for _ in range(2)]
    assert caches[0].numel() > 1 << 31
    for x, y in zip(caches, c["caches"]):
        x.view(torch.uint8)[-small:] = y.view(torch.uint8).cuda()
    d = Device(c)
    d.k, d.v = caches
    d.d = bgg.bgg_cache_describe("e4m3", pages * 2, page, hk, D)
    d.table = torch.where(d.table >= 0, d.table + pages * 2 - small, d.table)
    d.step()
    d.check()


def test_refusals_of_the_binding():
    c = case([(2, [5, 3])], hq=4, hk=2, D=64)
    d = Device(c)

    def go(**change):
        a = dict(table=d.table, lengths=d.n, starts=d.starts, shared=d.shared, q=d.q, out=d.out, ws=d.ws)
        a.update(change)
        bgg.bgg_shared_attention(d.d, d.k, d.v, a["table"], a["lengths"], a["starts"], a["shared"], a["q"], a["out"], a["ws"],
                                 scale=0.1)

    go()
    i32 = dict(dtype=torch.int32, device="cuda")
    for change in (dict(starts=d.starts.cpu()), dict(starts=d.starts.long()), dict(starts=None), dict(shared=None),
                   dict(shared=d.shared[:1]), dict(starts=torch.zeros(0, **i32)), dict(ws=d.ws[:100000]),
                   dict(starts=torch.zeros(4, **i32)), dict(lengths=d.n[:1]), dict(table=d.table[:1])):
        with pytest.raises((ValueError, bgg.BggError)):
            go(**change)
    go(table=d.table[:0], lengths=d.n[:0], starts=torch.zeros(1, **i32), shared=d.shared[:0], q=d.q[:0], out=d.out[:0])
