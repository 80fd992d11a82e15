"""Cases of the operators of a serving step on a paged cache: page tables and
slots built on the GPU from the lengths of the requests, rotary positions with
several axes, and the attention of sequences that share a long prefix.

`run` computes a case in plain torch (`own` false) or through the library's
entry points (`own` true); both take the state that `prepare` makes.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


def listed():
    return [
        # --- page tables and slots from the requests' lengths
        # one conversation, one more token: latency
        dict(name="assign_1", op="assign", B=1, rows=1, page=16, width=2048, new="one", cut=0.0, shared=0, spare=8),
        # a decode step of a serving batch
        dict(name="assign_64", op="assign", B=64, rows=64, page=16, width=2048, new="one", cut=0.0, shared=0, spare=64),
        # requests of very different kinds in one padded step: prompts, single tokens, some that end or give
        # rejected draft tokens back, behind a shared prefix
        dict(name="assign_300_mixed", op="assign", B=300, rows=70001, page=32, width=1024, new="mixed", cut=0.25, shared=9,
             spare=100),
        # the largest batch, long prompts, and too few free pages for the last of them
        dict(name="assign_4096_prompts", op="assign", B=4096, rows=1000000, page=64, width=256, new="prompt", cut=0.1,
             shared=0, spare=-300),
        # --- rotary positions with several axes, keys and values into the paged cache
        # one decoded token behind images: time, height and width
        dict(name="axes_1", op="axes", T=1, q_heads=48, kv_heads=8, head_dim=128, sections="16+24+24", arrangement="blocks",
             layout="half", dtype="f16", kv="f16", page=16, append=True),
        # video patches of several requests into an 8-bit cache, a quarter of the head rotated, axes in turn
        dict(name="axes_777_e4m3", op="axes", T=777, q_heads=24, kv_heads=4, head_dim=256, sections="11+11+10",
             arrangement="cyclic", layout="half", dtype="f16", kv="e4m3", page=64, append=True),
        # an image tower's patches: two axes, queries and keys as one row of heads, no cache
        dict(name="axes_9409_image", op="axes", T=9409, q_heads=32, kv_heads=16, head_dim=64, sections="16+16",
             arrangement="blocks", layout="interleaved", dtype="bf16", kv="bf16", page=16, append=False),
        # --- attention of one new token per sequence, behind prefixes that sequences share
        # four samples of one short prompt: latency
        dict(name="shared_4x500", op="shared", groups="4x32", own=60, q_heads=48, kv_heads=8, head_dim=128, dtype="f16",
             kv="f16", page=16, window=0, unused=0),
        # a serving batch behind one long system prompt, one slot of it unused
        dict(name="shared_16x8192", op="shared", groups="16x128", own=2000, q_heads=24, kv_heads=4, head_dim=256,
             dtype="bf16", kv="bf16", page=64, window=0, unused=1),
        # three prompts with groups of different sizes, a sliding window, the 8-bit cache
        dict(name="shared_groups_e4m3", op="shared", groups="7x200+1x900+40x511", own=700, q_heads=32, kv_heads=8,
             head_dim=64, dtype="f16", kv="e4m3", page=32, window=9001, unused=2),
        # many samples of one long document
        dict(name="shared_64x32768", op="shared", groups="64x512", own=300, q_heads=48, kv_heads=8, head_dim=128,
             dtype="f16", kv="f16", page=64, window=0, unused=0),
        # a large batch, two shared prompts of odd sizes
        dict(name="shared_256_bf16", op="shared", groups="157x333+99x257", own=200, q_heads=32, kv_heads=8,
             head_dim=128, dtype="bf16", kv="bf16", page=16, window=0, unused=5),
    ]


def _sections(c):
    """Pairs that each axis turns."""
    return [int(v) for v in c["sections"].split("+")]


def _groups(c):
    """(sequences, pages they share) of each group."""
    return [tuple(int(v) for v in g.split("x")) for g in c["groups"].split("+")]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["assign", "axes", "shared", "shared"])
    if op == "assign":
        B, page = _log(rng, 1, 4096), rng.choice([16, 32, 64, 128, 256])
        new = rng.choice(["one", "mixed", "prompt"])
        return dict(op=op, B=B, rows=B if new == "one" else _log(rng, B, 500000), page=page,
                    width=_log(rng, 2, min(4096, (1 << 22) // B)), new=new, cut=rng.choice([0.0, 0.0, 0.2, 0.5]),
                    shared=rng.choice([0, rng.randint(0, 20)]), spare=_log(rng, 1, 1000) * rng.choice([1, 1, -1]))
    q_heads, kv_heads = rng.choice([(48, 8), (24, 4), (32, 8), (32, 32), (8, 2), (16, 1), (12, 12), (40, 2), (7, 1)])
    head_dim = rng.choice([64, 96, 128, 192, 256])
    dtype = rng.choice(["f16", "bf16"])
    kv = rng.choice([dtype, dtype, "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "axes":
        pairs, n = rng.choice([head_dim // 2, head_dim // 4, head_dim // 8]), rng.choice([2, 3, 3, 4])
        cut = sorted(rng.sample(range(1, pairs), n - 1))
        sections = [b - a for a, b in zip([0] + cut, cut + [pairs])]
        arrangement = "blocks"
        if rng.random() < 0.4:  # in turn: as even as the pairs allow, the first axis has the rest
            sections = [pairs - (n - 1) * (pairs // n)] + [pairs // n] * (n - 1)
            arrangement = "cyclic"
        append = rng.random() < 0.7
        most = 18000000 // ((q_heads + 2 * kv_heads) * head_dim)
        return dict(op=op, T=_log(rng, 1, min(5000, most)), q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                    sections="+".join(map(str, sections)),
                    arrangement=arrangement, layout=rng.choice(["half", "interleaved"]), dtype=dtype, kv=kv, page=page,
                    append=append)
    B = _log(rng, 2, 128)
    n = rng.choice([1, 1, 2, min(5, B)])
    cut = sorted(rng.sample(range(1, B), n - 1))
    # (scores and widened values of the plain form stay within a few gigabytes)
    most = max(page, min(32768, (1 << 27) // (kv_heads * head_dim), (1 << 28) // (B * q_heads),
                         (1 << 33) // (B * q_heads * head_dim)))
    groups = [(b - a, _log(rng, 1, max(1, most // page))) for a, b in zip([0] + cut, cut + [B])]
    own_tokens = _log(rng, 1, max(1, min(3000, (1 << 26) // (B * kv_heads * head_dim))))
    longest = max(g[1] for g in groups) * page + own_tokens
    return dict(op=op, groups="+".join("%dx%d" % g for g in groups), own=own_tokens, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                kv=kv, page=page, window=rng.choice([0, 0, _log(rng, 1, longest)]), unused=rng.choice([0, 0, 1]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(0x0A551 + 7919 * seed)
    return g


def _randn(g, shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _requests(c, seed):
    """(tokens in the cache, new tokens) of each sequence; fewer than 0: given back.  The
    seed sets their order."""
    r = random.Random(c["B"] * 1000003 + c["rows"])
    ps, most, left = c["page"], c["width"] * c["page"], c["rows"]
    have, new = [], []
    for b in range(c["B"]):
        base = min(c["shared"], c["width"]) * ps
        n = base + _log(r, 1, max(1, most - base)) - 1
        others = c["B"] - 1 - b  # at least a token is left for each of them
        k = min(1, left)
        if c["new"] == "prompt" or (c["new"] == "mixed" and r.random() < 0.3):
            n = base
            k = min(_log(r, 1, max(1, 2 * c["rows"] // c["B"])), max(0, left - others), max(1, most - n))
        if r.random() < c["cut"]:
            k = -min(n, r.choice([n, r.randint(0, 8)]))  # it ends, or gives draft tokens back
            if r.random() < 0.1:
                k = -(1 << 31)
        left -= max(k, 0)
        have.append(n)
        new.append(k)
    order = list(range(c["B"]))
    random.Random(seed).shuffle(order)
    return [have[b] for b in order], [new[b] for b in order]


def _prepare_assign(c, seed):
    g, B, W, ps = _gen(seed), c["B"], c["width"], c["page"]
    have, new = _requests(c, seed)
    held = [-(-n // ps) for n in have]
    shared = min(c["shared"], W)
    need = sum(max(0, -(-(n + k) // ps) - h) for n, k, h in zip(have, new, held) if k > 0)
    free = max(1, need + c["spare"])
    capacity = shared + sum(max(0, h - shared) for h in held) + free
    order = torch.randperm(capacity, generator=g, device=DEV).to(torch.int32)
    held_t = torch.tensor(held, device=DEV)
    p = torch.arange(W, device=DEV)
    mine = (p >= shared) & (p < held_t[:, None])
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    at = shared + torch.cumsum(mine.flatten(), 0).view(B, W) - 1
    table = torch.where(mine, order[at.clamp(min=0)], table)
    table = torch.where((p < shared) & (p < held_t[:, None]), order[p.clamp(max=max(shared - 1, 0))], table)
    # a window has left the first pages of some sequences behind
    if c["cut"] and not shared:
        gone = torch.rand((B, 1), generator=g, device=DEV) < 0.2
        table = torch.where(gone & (p < held_t[:, None] // 3), torch.full_like(table, -1), table)
    free_pages = torch.full((capacity,), -1, dtype=torch.int32, device=DEV)
    free_pages[:free] = order[capacity - free:]
    T = c["rows"]
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(c=c, lengths=torch.tensor(have, **i32), counts=torch.tensor(new, dtype=torch.int64).to(torch.int32).to(DEV),
                table=table.contiguous(), table_start=table.clone(), free=free_pages, free_start=free_pages.clone(),
                count=torch.tensor([free], **i32), shared=torch.full((B,), shared, **i32) if c["shared"] else None,
                pages=capacity, lengths_out=torch.zeros(B, **i32), count_out=torch.zeros(1, **i32),
                past=torch.zeros(B, **i32), starts=torch.zeros(B + 1, **i32), positions=torch.zeros(T, **i32),
                slots=torch.zeros(T, dtype=torch.int64, device=DEV))


def _axis_of_pair(sections, arrangement):
    """The axis whose position turns each pair."""
    n, pairs = len(sections), sum(sections)
    if arrangement == "blocks":
        return [a for a, s in enumerate(sections) for _ in range(s)]
    return [i % n if i < n * sections[i % n] else 0 for i in range(pairs)]


def _prepare_axes(c, seed):
    g, T, dt = _gen(seed), c["T"], TYPES[c["dtype"]]
    Hq, Hk, D, ps, A = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], len(_sections(c))
    pairs = sum(_sections(c))
    heads = Hq + 2 * Hk if c["append"] else Hq
    row = _randn(g, (T, heads * D), 1.0, dt)  # q, k and v of one grouped product
    pages = -(-T // ps) + 3 if c["append"] else 1
    slots = (torch.randperm(pages, generator=g, device=DEV)[:, None] * ps + torch.arange(ps, device=DEV)).view(-1)[:T]
    if T > 4 and c["append"]:  # an unused row of the batch
        slots = slots.clone()
        slots[T // 2] = -1
    # patches of images up to a few hundred patches wide, far into their sequence
    side = max(1, math.isqrt(T))
    t = torch.arange(T, device=DEV)
    first = int(torch.randint(0, 200000, (1,), generator=g, device=DEV).item())
    rows = [first + t // (side * side), first + (t // side) % side, first + t % side, first + t]
    rows = rows[1:3] if A == 2 else rows[:A]
    st = dict(c=c, row=row, pos=torch.stack(rows).to(torch.int32).contiguous(), slots=slots.to(torch.int64).contiguous(),
              axes=torch.tensor(_axis_of_pair(_sections(c), c["arrangement"]), dtype=torch.uint8, device=DEV),
              magnitude=1.0, pages=pages, q_out=torch.empty((T, Hq * D), dtype=dt, device=DEV), k_scale=None, v_scale=None)
    i = torch.arange(0, 2 * pairs, 2, dtype=torch.float64, device=DEV)
    st["freqs"] = (1e6 ** (-i / (2 * pairs))).float()
    if c["append"]:
        for n in ("k_cache", "v_cache"):
            st[n] = _randn(g, (pages, Hk, ps, D), 1.0, torch.float32).to(TYPES[c["kv"]])
            st[n + "_start"] = st[n].clone()
        if c["kv"] == "e4m3":
            st["k_scale"], st["v_scale"] = (torch.rand((Hk,), generator=g, device=DEV) * 0.02 + 0.01 for _ in range(2))
    return st


def _sequences(c):
    """(group, tokens) of each sequence: its group's prefix and 1..own tokens of its
    own, spread on a log scale; unused slots have no tokens."""
    r = random.Random(len(_groups(c)) * 1000003 + c["own"])
    n = [(k, pages * c["page"] + _log(r, 1, c["own"])) for k, (members, pages) in enumerate(_groups(c))
         for _ in range(members)]
    for b in r.sample(range(len(n)), min(c["unused"], len(n) - 1)):
        n[b] = (n[b][0], 0)
    return n


def _prepare_shared(c, seed):
    g, dt, kt = _gen(seed), TYPES[c["dtype"]], TYPES[c["kv"]]
    Hq, Hk, D, ps = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    seqs = _sequences(c)
    B = len(seqs)
    prefix = [pages for _, pages in _groups(c)]
    mine = [max(0, -(-n // ps) - prefix[k]) for k, n in seqs]
    width = max(prefix[k] + m for (k, _), m in zip(seqs, mine))
    pages = sum(prefix) + sum(mine) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at, shared = 0, []
    for k in prefix:
        shared.append(order[at: at + k])
        at += k
    starts = [0]
    for members, _ in _groups(c):
        starts.append(starts[-1] + members)
    for b, (k, n) in enumerate(seqs):
        table[b, : prefix[k]] = shared[k]
        table[b, prefix[k]: prefix[k] + mine[b]] = order[at: at + mine[b]]
        at += mine[b]
    st = dict(c=c, table=table.to(DEV), lengths=torch.tensor([n for _, n in seqs], dtype=torch.int32, device=DEV),
              group_starts=torch.tensor(starts, dtype=torch.int32, device=DEV), starts=starts,
              shared_pages=torch.tensor([prefix[k] for k, _ in seqs], dtype=torch.int32, device=DEV), pages=pages,
              widths=[max(mine[a:b]) for a, b in zip(starts, starts[1:])],
              q=_randn(g, (B, Hq * D), 1.5, dt), out=torch.empty((B, Hq * D), dtype=dt, device=DEV),
              lse=torch.empty((B, Hq), dtype=torch.float32, device=DEV), scale=D ** -0.5)
    for name in ("k", "v"):
        cache = torch.empty((pages, Hk, ps, D), dtype=kt, device=DEV)
        step = max(1, (1 << 26) // (Hk * ps * D))
        for p in range(0, pages, step):
            part = cache[p: p + step]
            part.copy_(torch.randn(part.shape, generator=g, device=DEV) * (50.0 if c["kv"] == "e4m3" else 1.0))
        st[name + "_cache"] = cache
        st[name + "_scale"] = torch.rand((Hk,), generator=g, device=DEV) * 0.01 + 0.015 if c["kv"] == "e4m3" else None
    return st


def prepare(case, seed):
    return {"assign": _prepare_assign, "axes": _prepare_axes, "shared": _prepare_shared}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
_workspaces = {}


def _workspace(kind, nbytes):
    """The program's workspace for one kind of call: zero-filled once, kept,
    replaced by a larger one where a call needs more."""
    w = _workspaces.get(kind)
    if w is None or w.numel() < nbytes:
        w = _workspaces[kind] = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=DEV)
    return w


def _own_assign(st):
    import bit_gemv_gemm_amd as bgg
    if "cache" not in st:
        st["cache"] = bgg.bgg_cache_describe("f16", st["pages"], st["c"]["page"], 8, 128)
    bgg.bgg_cache_assign(st["cache"], st["lengths"], st["counts"], st["table"], st["free"], st["count"], st["lengths_out"],
                         st["count_out"], st["past"], st["starts"], st["positions"], st["slots"],
                         shared_pages=st["shared"])
    return _assigned(st)


def _own_axes(st):
    import bit_gemv_gemm_amd as bgg
    c = st["c"]
    if "cache" not in st:
        st["cache"] = bgg.bgg_cache_describe(c["kv"], st["pages"], c["page"], c["kv_heads"], c["head_dim"])
        nq, nk = c["q_heads"] * c["head_dim"], c["kv_heads"] * c["head_dim"]
        st["q"] = st["row"][:, :nq]
        st["k"], st["v"] = (st["row"][:, nq:nq + nk], st["row"][:, nq + nk:]) if c["append"] else (None, None)
    if not c["append"]:
        bgg.bgg_rotary_append_axes(st["cache"], None, None, st["pos"], st["axes"], None, st["freqs"], q=st["q"],
                                   q_out=st["q_out"], layout=c["layout"], magnitude=st["magnitude"])
        return {"q": st["q_out"]}
    bgg.bgg_rotary_append_axes(st["cache"], st["k_cache"], st["v_cache"], st["pos"], st["axes"], st["slots"], st["freqs"],
                               q=st["q"], q_out=st["q_out"], k=st["k"], v=st["v"], layout=c["layout"],
                               magnitude=st["magnitude"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}


def _own_shared(st):
    import bit_gemv_gemm_amd as bgg
    c = st["c"]
    if "cache" not in st:
        st["cache"] = bgg.bgg_cache_describe(c["kv"], st["pages"], c["page"], c["kv_heads"], c["head_dim"])
        st["need"] = bgg.bgg_shared_attention_workspace_size(st["cache"], c["q_heads"], st["q"].shape[0])
    bgg.bgg_shared_attention(st["cache"], st["k_cache"], st["v_cache"], st["table"], st["lengths"], st["group_starts"],
                             st["shared_pages"], st["q"], st["out"], _workspace("attention", st["need"]),
                             scale=st["scale"], window=c["window"], lse=st["lse"], k_scale=st["k_scale"],
                             v_scale=st["v_scale"])
    return {"out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _assigned(st):
    return {"table": st["table"], "lengths": st["lengths_out"], "free": st["free"], "count": st["count_out"],
            "past": st["past"], "starts": st["starts"], "positions": st["positions"], "slots": st["slots"]}


def _plain_assign(st):
    c = st["c"]
    ps, W, T, capacity = c["page"], c["width"], c["rows"], st["free"].numel()
    n = st["lengths"].long().clamp(0, W * ps)
    k = st["counts"].long()
    low = st["shared"].long().clamp(0, W) * ps if st["shared"] is not None else torch.zeros_like(n)
    past = torch.where(k < 0, torch.minimum(n, torch.maximum(n + k, low)), n)
    k = k.clamp(min=0)
    held = lambda v: (v + ps - 1) // ps
    p = torch.arange(W, device=DEV)
    # pages given back: the last sequence's last page first
    back = (p >= held(past)[:, None]) & (p < held(n)[:, None]) & (st["table"] >= 0) & (st["table"] < st["pages"])
    back, page = back.flatten().flip(0), st["table"].flatten().flip(0)
    at = st["count"].long().clamp(0, capacity) + torch.cumsum(back, 0) - 1
    at = torch.where(back & (at < capacity), at, capacity)
    free = torch.cat([st["free"], st["free"][:1]])
    free[at] = page
    free = free[:-1]
    have = (st["count"].long().clamp(0, capacity) + back.sum()).clamp(max=capacity)
    # pages taken: from the top, in order of the sequences
    end = torch.cumsum(k, 0)
    fits = (end <= T) & (past + k <= W * ps)
    need = torch.where(fits, held(past + k) - held(past), 0)
    upto = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (upto <= have))
    taken = torch.where(served & (need > 0), upto, 0).amax()
    new = (p >= held(past)[:, None]) & (p < held(past + k)[:, None]) & served[:, None]
    top = have - 1 - ((upto - need)[:, None] + p - held(past)[:, None])
    table = torch.where(new, free[top.clamp(0, capacity - 1)], st["table"])
    # the rows of the new tokens
    start = end - k
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(end, t, right=True)
    real = b < c["B"]
    b = b.clamp(max=c["B"] - 1)
    real = real & served[b]
    pos = past[b] + t - start[b]
    cell = table[b, torch.where(real, pos // ps, 0)].long()
    ok = real & (cell >= 0) & (cell < st["pages"])
    st["table"].copy_(table)
    st["free"].copy_(free)
    st["lengths_out"].copy_(torch.where(served, past + k, past))
    st["count_out"].copy_((have - taken).view(1))
    st["past"].copy_(past)
    st["starts"].copy_(torch.cat([torch.zeros_like(end[:1]), end]).clamp(max=T))
    st["positions"].copy_(torch.where(real, pos, 0))
    st["slots"].copy_(torch.where(ok, cell * ps + pos % ps, -1))
    return _assigned(st)


def _turn(x, cos, sin, layout):
    """x [T, H, D] with its first 2 * pairs values rotated by pairs."""
    n = cos.shape[-1]
    r, rest = x[..., : 2 * n], x[..., 2 * n:]
    if layout == "half":
        a, b = r[..., :n], r[..., n:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def _plain_axes(st):
    c, T = st["c"], st["c"]["T"]
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    row = st["row"].float().view(T, -1, D)
    angle = st["pos"].double()[st["axes"].long()].t() * st["freqs"].double()
    cos, sin = (f(angle)[:, None] * st["magnitude"] for f in (torch.cos, torch.sin))
    cos, sin = cos.float(), sin.float()
    q = _turn(row[:, :Hq], cos, sin, c["layout"])
    got = {"q": q.to(TYPES[c["dtype"]]).view(T, Hq * D)}
    if not c["append"]:
        return got
    k = _turn(row[:, Hq:Hq + Hk], cos, sin, c["layout"])
    v = row[:, Hq + Hk:]
    if st["k_scale"] is not None:
        k = (k / st["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / st["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    # tokens without a slot write into a spare page behind the cache
    slot = torch.where(st["slots"] < 0, st["pages"] * c["page"], st["slots"])
    for name, x in (("k", k), ("v", v)):
        cache = st[name + "_cache"]
        bits = torch.uint8 if c["kv"] == "e4m3" else torch.int16
        cells = cache.view(bits).transpose(1, 2).reshape(-1, Hk, D)
        cells = torch.cat([cells, cells[:1]])
        cells[slot] = x.to(cache.dtype).view(bits)
        cells = cells[:-1].view(st["pages"], c["page"], Hk, D).transpose(1, 2)
        cache.view(bits).copy_(cells)
        got[name] = cache
    return got


def _plain_shared(st):
    c = st["c"]
    Hq, Hk, D, ps = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    G = Hq // Hk
    zero = torch.zeros((), device=DEV)
    outs, lses = [], []
    for (members, prefix), a, width in zip(_groups(c), st["starts"], st["widths"]):
        rows = slice(a, a + members)
        n = st["lengths"][rows][:, None]
        q = st["q"][rows].float().view(members, Hk, G, D) * st["scale"]
        if st["k_scale"] is not None:
            q = q * st["k_scale"][:, None, None]

        def seen_of(t):
            return (t < n) & (t >= n - c["window"]) if c["window"] else t < n

        # the prefix: its keys and values once, against every row of the group
        pages = st["table"][a, :prefix].long()
        L = prefix * ps
        see = seen_of(torch.arange(L, device=DEV))
        k = st["k_cache"][pages].transpose(0, 1).reshape(Hk, L, D).float().transpose(1, 2).contiguous()
        s = q.transpose(0, 1).reshape(Hk, members * G, D) @ k
        s = s.view(Hk, members, G, L).masked_fill(~see[:, None, :], -math.inf)
        del k
        # each sequence's own tokens
        t = L + torch.arange(width * ps, device=DEV)
        see_own = seen_of(t)
        table = st["table"][rows, prefix:prefix + width].clamp(min=0).long()
        k = st["k_cache"][table].transpose(1, 2).reshape(members, Hk, width * ps, D).float().transpose(2, 3).contiguous()
        s_own = (q @ k).masked_fill(~see_own[:, None, None, :], -math.inf)  # [members, Hk, G, own]
        del k
        m = torch.maximum(s.amax(-1), s_own.amax(-1).transpose(0, 1)) if width else s.amax(-1)  # [Hk, members, G]
        m0 = torch.where(m == -math.inf, zero, m)
        s = torch.exp(s - m0[..., None])
        s_own = torch.exp(s_own - m0.transpose(0, 1)[..., None])
        total = s.sum(-1).transpose(0, 1) + s_own.sum(-1)  # [members, Hk, G]
        v = st["v_cache"][pages].transpose(0, 1).reshape(Hk, L, D).float()
        o = (s.view(Hk, members * G, L) @ v).view(Hk, members, G, D).transpose(0, 1)
        del v, s
        v = st["v_cache"][table].transpose(1, 2).reshape(members, Hk, width * ps, D).float()
        o = o + s_own @ torch.where(see_own[:, None, :, None], v, zero)
        o = o / torch.where(total == 0, torch.ones_like(total), total)[..., None]
        if st["v_scale"] is not None:
            o = o * st["v_scale"][:, None, None]
        outs.append(o.reshape(members, Hq * D).to(TYPES[c["dtype"]]))
        lses.append((torch.log(total) + m.transpose(0, 1)).reshape(members, Hq))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"assign": _own_assign, "axes": _own_axes, "shared": _own_shared}[op](state)
    return {"assign": _plain_assign, "axes": _plain_axes, "shared": _plain_shared}[op](state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "assign":
        have, new = _requests(c, 0)
        ps = c["page"]
        moved = sum(-(-(n + k) // ps) + (-n // ps) if k > 0 else min(-(-n // ps), -(k // ps)) for n, k in zip(have, new) if k)
        return {"bytes": 20 * c["B"] + 12 * c["rows"] + 8 * moved, "flops": 4 * c["B"] + 4 * c["rows"]}
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    kb = 1 if c["kv"] == "e4m3" else 2
    if c["op"] == "axes":
        T, pairs, A = c["T"], sum(_sections(c)), len(_sections(c))
        b = T * (4 * D * Hq + 4 * A) + 5 * pairs + c["append"] * T * (4 * Hk * D + 2 * Hk * D * kb + 8)
        return {"bytes": b, "flops": T * (Hq + c["append"] * Hk) * pairs * 6}
    seqs = _sequences(c)
    rows, cached = 0, 0
    for k, (members, pages) in enumerate(_groups(c)):
        L = pages * c["page"]
        mine = [n for kk, n in seqs if kk == k]
        seen = [(max(0, n - c["window"]) if c["window"] else 0, n) for n in mine]
        rows += sum(n - lo for lo, n in seen)
        cached += sum(max(0, n - max(lo, L)) for lo, n in seen) + max([0] + [L - min(lo, L) for lo, n in seen if n])
    B = len(seqs)
    b = 2 * cached * Hk * D * kb + 4 * B * Hq * D + 4 * B * (Hq + 1) + 4 * (cached // c["page"])
    return {"bytes": b, "flops": 4 * rows * Hq * D}


def _exact_assign(c, st):
    """A stack of free pages, one sequence after the other."""
    ps, W, T = c["page"], c["width"], c["rows"]
    n, k = st["lengths"].tolist(), st["counts"].tolist()
    table, stack = st["table_start"].tolist(), st["free_start"].tolist()
    capacity, top = len(stack), st["count"].item()
    low = (st["shared"].tolist() if st["shared"] is not None else [0] * c["B"])
    past, after = list(n), list(n)
    for b in reversed(range(c["B"])):
        if k[b] < 0:
            past[b] = after[b] = min(n[b], max(n[b] + k[b], low[b] * ps))
            for p in reversed(range(math.ceil(past[b] / ps), math.ceil(n[b] / ps))):
                if 0 <= table[b][p] < st["pages"] and top < capacity:
                    stack[top] = table[b][p]
                    top += 1
    starts, positions, slots = [0], [0] * T, [-1] * T
    row, closed = 0, False
    for b in range(c["B"]):
        new, first = max(k[b], 0), row
        row += new
        starts.append(min(row, T))
        if row > T or past[b] + new > W * ps:
            continue
        wanted = range(math.ceil(past[b] / ps), math.ceil((past[b] + new) / ps))
        if len(wanted) and (closed or len(wanted) > top):
            closed = True  # nor does any after it get pages
            continue
        for p in wanted:
            top -= 1
            table[b][p] = stack[top]
        after[b] = past[b] + new
        for i in range(new):
            at = past[b] + i
            positions[first + i] = at
            page = table[b][at // ps]
            slots[first + i] = page * ps + at % ps if 0 <= page < st["pages"] else -1
    i32 = dict(dtype=torch.int32, device=DEV)
    return {"table": torch.tensor(table, **i32), "lengths": torch.tensor(after, **i32), "free": torch.tensor(stack, **i32),
            "count": torch.tensor([top], **i32), "past": torch.tensor(past, **i32), "starts": torch.tensor(starts, **i32),
            "positions": torch.tensor(positions, **i32), "slots": torch.tensor(slots, dtype=torch.int64, device=DEV)}


def _exact_axes(c, st):
    T, Hq, Hk, D = c["T"], c["q_heads"], c["kv_heads"], c["head_dim"]
    pairs = sum(_sections(c))
    z = st["row"].double().view(T, -1, D)
    turning = Hq + Hk if c["append"] else Hq
    pos = torch.empty((T, pairs), dtype=torch.float64, device=DEV)
    for i, a in enumerate(_axis_of_pair(_sections(c), c["arrangement"])):
        pos[:, i] = st["pos"][a].double()
    turn = torch.polar(torch.full((T, 1, pairs), st["magnitude"], dtype=torch.float64, device=DEV),
                       (pos * st["freqs"].double())[:, None, :])
    first = torch.arange(pairs, device=DEV) * (1 if c["layout"] == "half" else 2)
    second = first + (pairs if c["layout"] == "half" else 1)
    w = torch.complex(z[:, :turning, first], z[:, :turning, second]) * turn
    z[:, :turning, first], z[:, :turning, second] = w.real, w.imag
    got = {"q": z[:, :Hq].reshape(T, Hq * D)}
    if not c["append"]:
        return got
    kept = st["slots"] >= 0
    page, cell = st["slots"][kept] // c["page"], st["slots"][kept] % c["page"]
    for name, x in (("k", z[:, Hq:Hq + Hk]), ("v", z[:, Hq + Hk:])):
        if c["kv"] == "e4m3":
            x = torch.clamp(x / st[name + "_scale"].double()[:, None], -E4M3_MAX, E4M3_MAX)
        cache = st[name + "_cache_start"].double()
        cache[page, :, cell] = x[kept]
        got[name] = cache
    return got


def _exact_shared(c, st):
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    seqs = _sequences(c)
    B = len(seqs)
    if sum(n for _, n in seqs) * Hk * D > 1 << 33:
        return None
    out = torch.zeros((B, Hk, Hq // Hk, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hk, Hq // Hk), -math.inf, dtype=torch.float64, device=DEV)
    q = st["q"].double().view(B, Hk, -1, D)
    for b, (_, n) in enumerate(seqs):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        t = torch.arange(lo, n, device=DEV)
        page, cell = st["table"][b].long()[t // c["page"]], t % c["page"]
        for h in range(Hk):
            k = st["k_cache"][page, h, cell].double()
            v = st["v_cache"][page, h, cell].double()
            if c["kv"] == "e4m3":
                k, v = k * st["k_scale"][h].double(), v * st["v_scale"][h].double()
            s = (q[b, h] @ k.t().contiguous()) * st["scale"]
            lse[b, h] = torch.logsumexp(s, -1)
            out[b, h] = torch.exp(s - lse[b, h][:, None]) @ v
    return {"out": out.view(B, Hq * D), "lse": lse.view(B, Hq)}


def exact(case, seed):
    return {"assign": _exact_assign, "axes": _exact_axes, "shared": _exact_shared}[case["op"]](case, prepare(case, seed))
