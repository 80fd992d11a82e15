"""Cases of the operators around the ternary products of a decoder layer:
the products with an epilogue, rotary positions with the append to a paged
key/value cache, and the attention of one new token over that cache.

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
        # --- products with an epilogue: y = act(W x + bias) * mul + residual
        # the down projection of one decoded token, added to the residual stream
        dict(name="product_down_1", op="product", fmt="PQ2_0", M=1, N=5120, K=17408,
             act="none", bias=False, mul=False, residual=True, rotate=True),
        # the gate projection of a decode batch: silu(gate) times the up projection
        dict(name="product_gate_16", op="product", fmt="PTQ1_0", M=16, N=17408, K=5120,
             act="silu", bias=False, mul=True, residual=False, rotate=True),
        # a short prompt's tail (77 tokens), odd row count, bias and gelu
        dict(name="product_prompt_77", op="product", fmt="PTQ1_0", M=77, N=6100, K=5120,
             act="gelu", bias=True, mul=False, residual=True, rotate=False),
        # the gate projection of a long prompt
        dict(name="product_gate_4096", op="product", fmt="PQ2_0", M=4096, N=17408, K=5120,
             act="silu", bias=False, mul=True, residual=False, rotate=False),
        # --- rotary positions, keys and values into the paged cache
        # one decoded token far into its context
        dict(name="rotary_1", op="rotary", T=1, q_heads=48, kv_heads=8, head_dim=128, rotary_dim=128,
             layout="half", dtype="f16", kv="f16", page=16, far=260000),
        # a decode batch, a quarter of the head rotated, 8-bit cache
        dict(name="rotary_16_e4m3", op="rotary", T=16, q_heads=24, kv_heads=4, head_dim=256, rotary_dim=64,
             layout="interleaved", dtype="f16", kv="e4m3", page=64, far=30000),
        # a prompt, odd length
        dict(name="rotary_4095", op="rotary", T=4095, q_heads=48, kv_heads=8, head_dim=128, rotary_dim=128,
             layout="half", dtype="bf16", kv="bf16", page=64, far=0),
        # --- attention of one new token per sequence over the paged cache
        # a single short conversation: latency
        dict(name="attention_1x500", op="attention", B=1, L=500, q_heads=48, kv_heads=8, head_dim=128,
             dtype="f16", kv="f16", page=16, window=0, ragged=False),
        # a serving batch of ragged lengths, one slot of it unused
        dict(name="attention_16_ragged", op="attention", B=16, L=8000, q_heads=24, kv_heads=4, head_dim=256,
             dtype="bf16", kv="bf16", page=64, window=0, ragged=True),
        # many sequences with a sliding window, one key head per query head
        dict(name="attention_64_window", op="attention", B=64, L=3001, q_heads=32, kv_heads=32, head_dim=64,
             dtype="f16", kv="f16", page=32, window=1000, ragged=True),
        # one sequence at the full context of the 27B-class model
        dict(name="attention_1x262144", op="attention", B=1, L=262144, q_heads=48, kv_heads=8, head_dim=128,
             dtype="f16", kv="f16", page=64, window=0, ragged=False),
        # a long-context batch on the 8-bit cache
        dict(name="attention_16x32768_e4m3", op="attention", B=16, L=32768, q_heads=48, kv_heads=8, head_dim=128,
             dtype="f16", kv="e4m3", page=128, window=0, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "rotary", "attention"])
    if op == "product":
        small = rng.random() < 0.5
        fmt = rng.choice(["PQ2_0", "PTQ1_0", "Q1_0", "Q2_0_G64"] if small else ["PQ2_0", "PTQ1_0"])
        return dict(op=op, fmt=fmt, M=rng.randint(1, 16) if small else _log(rng, 17, 2000),
                    N=_log(rng, 200, 17408), K=128 * _log(rng, 4, 100),
                    act=rng.choice(["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]),
                    bias=rng.random() < 0.5, mul=rng.random() < 0.5, residual=rng.random() < 0.5,
                    rotate=small)
    q_heads, kv_heads = rng.choice([(48, 8), (24, 4), (32, 8), (32, 32), (8, 2), (16, 1), (12, 12), (40, 2), (7, 1)])
    head_dim = rng.choice([64, 96, 128, 192, 256])
    dtype = rng.choice(["f16", "bf16"])
    kv = rng.choice([dtype, dtype, "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "rotary":
        return dict(op=op, T=_log(rng, 1, 3000), q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                    rotary_dim=rng.choice([head_dim, head_dim // 2, head_dim // 4]),
                    layout=rng.choice(["half", "interleaved"]), dtype=dtype, kv=kv, page=page,
                    far=_log(rng, 1, 1000000))
    B = _log(rng, 1, 64)
    most = max(1, min(65536, (1 << 27) // (B * kv_heads * head_dim)))
    L = _log(rng, 1, most)
    return dict(op=op, B=B, L=L, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, kv=kv,
                page=page, window=rng.choice([0, 0, _log(rng, 1, L)]), ragged=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(0x5EED0 + 7919 * seed)
    return g


def _randn(g, shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _scale_group(fmt):
    return 64 if fmt == "Q2_0_G64" else 128


def _row_bytes(fmt, t):
    """The canonical row stream of weights t, int8 [N, K]."""
    N, K = t.shape
    if fmt == "Q1_0":
        bits = (t.view(N, K // 8, 8) > 0).to(torch.int32)
        return (bits << torch.arange(8, device=DEV, dtype=torch.int32)).sum(-1).to(torch.uint8)
    c = t.to(torch.int32) + 1
    if fmt == "PTQ1_0":
        pad = -K % 5
        c = torch.cat([c, torch.ones((N, pad), dtype=torch.int32, device=DEV)], 1) if pad else c
        p = torch.tensor([1, 3, 9, 27, 81], dtype=torch.int32, device=DEV)
        return (c.view(N, -1, 5) * p).sum(-1).to(torch.uint8)
    p = torch.tensor([1, 4, 16, 64], dtype=torch.int32, device=DEV)
    return (c.view(N, -1, 4) * p).sum(-1).to(torch.uint8)


def _pack(fmt, t, s):
    """The packed buffer of bgg.h: 16-byte chunks and scales of 64-row tiles,
    then 8192 zero bytes."""
    rows = _row_bytes(fmt, t)
    N, nb = rows.shape
    tiles, chunks = -(-N // 64), -(-nb // 16)
    zero = {"PTQ1_0": 121, "Q1_0": 0}.get(fmt, 0x55)
    full = torch.full((tiles * 64, chunks * 16), zero, dtype=torch.uint8, device=DEV)
    full[:N, :nb] = rows
    trits = full.view(tiles, 64, chunks, 16).transpose(1, 2).reshape(-1)
    sc = torch.zeros((tiles * 64, s.shape[1]), dtype=torch.float16, device=DEV)
    sc[:N] = s
    sc = sc.view(tiles, 64, -1).transpose(1, 2).reshape(-1).view(torch.uint8)
    gap = torch.zeros(-trits.numel() % 256, dtype=torch.uint8, device=DEV)
    return torch.cat([trits, gap, sc, torch.zeros(8192, dtype=torch.uint8, device=DEV)])


def _prepare_product(c, seed):
    g, N, K, M = _gen(seed), c["N"], c["K"], c["M"]
    u = torch.rand((N, K), generator=g, device=DEV)
    # trits with 38 % zeros (signs for Q1_0), scales in [0.005, 0.05]
    if c["fmt"] == "Q1_0":
        t = torch.where(u < 0.5, -1, 1).to(torch.int8)
    else:
        t = (u > 0.69).to(torch.int8) - (u < 0.31).to(torch.int8)
    grp = _scale_group(c["fmt"])
    s = (torch.rand((N, K // grp), generator=g, device=DEV) * 0.045 + 0.005).to(torch.float16)
    x = _randn(g, (M, K))
    st = dict(c=c, x=x, y=torch.empty((M, N), dtype=torch.float16, device=DEV), packed=_pack(c["fmt"], t, s),
              # the matrix as a program without packed weights keeps it
              W=(t.view(N, K // grp, grp).float() * s.float()[:, :, None]).view(N, K), trits=t, scales=s)
    y_size = 0.025 * math.sqrt(0.62 * K)
    st["bias"] = _randn(g, (N,), y_size) if c["bias"] else None
    st["mul"] = _randn(g, (M, N), 1.0) if c["mul"] else None
    st["residual"] = _randn(g, (M, N), y_size) if c["residual"] else None
    h = torch.ones((1, 1), device=DEV)
    while h.shape[0] < 128:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    st["H"] = h.contiguous()
    return st


def _frequencies(rotary_dim):
    """Radians per position, float32 [rotary_dim / 2]."""
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=DEV)
    return (1e6 ** (-i / rotary_dim)).float()


def _prepare_rotary(c, seed):
    g, T, dt = _gen(seed), c["T"], TYPES[c["dtype"]]
    Hq, Hk, D, ps = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    row = _randn(g, (T, (Hq + 2 * Hk) * D), 1.0, dt)  # q, k and v of one grouped product
    pages = -(-T // ps) + 3
    slots = (torch.randperm(pages, generator=g, device=DEV)[:, None] * ps + torch.arange(ps, device=DEV)).view(-1)[:T]
    if c["far"]:  # tokens of different sequences, anywhere in their contexts
        pos = torch.randint(0, c["far"] + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
        if T > 4:  # an unused slot of the batch
            slots = slots.clone()
            slots[T // 2] = -1
    else:
        pos = torch.arange(T, dtype=torch.int32, device=DEV)
    st = dict(c=c, row=row, pos=pos, slots=slots.to(torch.int64).contiguous(), freqs=_frequencies(c["rotary_dim"]),
              magnitude=1.0625, pages=pages, q_out=torch.empty((T, Hq * D), dtype=dt, device=DEV))
    for n in ("k_cache", "v_cache"):
        st[n] = _randn(g, (pages, Hk, ps, D), 1.0, torch.float32).to(TYPES[c["kv"]])
        st[n + "_start"] = st[n].clone()
    st["k_scale"] = torch.rand((Hk,), generator=g, device=DEV) * 0.02 + 0.01 if c["kv"] == "e4m3" else None
    st["v_scale"] = torch.rand((Hk,), generator=g, device=DEV) * 0.02 + 0.01 if c["kv"] == "e4m3" else None
    return st


def _lengths(c):
    """Tokens of each sequence: all L, or spread over 1..L on a log scale with
    the longest L and, in a batch of four or more, one unused slot."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        return [L] * B
    r = random.Random(B * 1000003 + L)
    n = [_log(r, 1, L) for _ in range(B)]
    n[r.randrange(B)] = L
    if B >= 4:
        n[(n.index(L) + 1) % B] = 0
    return n


def _prepare_attention(c, seed):
    g, dt, kt = _gen(seed), TYPES[c["dtype"]], TYPES[c["kv"]]
    B, Hq, Hk, D, ps = c["B"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    n = _lengths(c)
    need = [-(-v // ps) for v in n]
    width, pages = max(max(need), 1), sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, : need[b]] = torch.tensor(order[at: at + need[b]], dtype=torch.int32)
        at += need[b]
    st = dict(c=c, table=table.to(DEV), lengths=torch.tensor(n, dtype=torch.int32, device=DEV), pages=pages,
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
    return {"product": _prepare_product, "rotary": _prepare_rotary, "attention": _prepare_attention}[case["op"]](case, seed)


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


def _own_product(st):
    import bit_gemv_gemm_amd as bgg
    c, M = st["c"], st["c"]["M"]
    gemv = M <= bgg.BGG_MAX_GEMV_M
    if "desc" not in st:
        st["desc"] = bgg.bgg_describe(c["fmt"], c["N"], c["K"])
        st["need"] = (bgg.bgg_gemv_workspace_size if gemv else bgg.bgg_gemm_workspace_size)(st["desc"], M)
    call = bgg.bgg_ternary_gemv_epilogue if gemv else bgg.bgg_ternary_gemm_epilogue
    call(st["desc"], st["packed"], st["x"], st["y"], M, bgg.BGG_ROTATE_INPUT if c["rotate"] else 0,
         _workspace("gemv" if gemv else "gemm", st["need"]), activation=c["act"], bias=st["bias"], mul=st["mul"],
         residual=st["residual"])
    return {"y": st["y"]}


def _own_rotary(st):
    import bit_gemv_gemm_amd as bgg
    c = st["c"]
    if "cache" not in st:
        st["cache"] = bgg.bgg_cache_describe(c["kv"], st["pages"], c["page"], c["kv_heads"], c["head_dim"])
        nq, nk = c["q_heads"] * c["head_dim"], c["kv_heads"] * c["head_dim"]
        st["q"], st["k"], st["v"] = st["row"][:, :nq], st["row"][:, nq:nq + nk], st["row"][:, nq + nk:]
    bgg.bgg_rotary_append(st["cache"], st["k_cache"], st["v_cache"], st["pos"], st["slots"], st["freqs"],
                          q=st["q"], q_out=st["q_out"], k=st["k"], v=st["v"], layout=c["layout"],
                          magnitude=st["magnitude"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}


def _own_attention(st):
    import bit_gemv_gemm_amd as bgg
    c = st["c"]
    if "cache" not in st:
        st["cache"] = bgg.bgg_cache_describe(c["kv"], st["pages"], c["page"], c["kv_heads"], c["head_dim"])
        st["need"] = bgg.bgg_attention_workspace_size(st["cache"], c["q_heads"], c["B"])
    bgg.bgg_paged_attention(st["cache"], st["k_cache"], st["v_cache"], st["table"], st["lengths"], st["q"], st["out"],
                            _workspace("attention", st["need"]), scale=st["scale"], window=c["window"], lse=st["lse"],
                            k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _activate(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "relu2":
        return torch.where(v < 0, torch.zeros_like(v), v) ** 2
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def _plain_product(st):
    c = st["c"]
    x = st["x"].float()
    if c["rotate"]:
        x = (x.view(-1, 128) @ st["H"]).view(x.shape) * (1 / math.sqrt(128))
    y = x @ st["W"].t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _activate(y, c["act"])
    if st["mul"] is not None:
        y = y * st["mul"].float()
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"y": y.to(torch.float16)}


def _turn(x, cos, sin, rotary_dim, layout):
    """x [T, H, D] with its first rotary_dim values rotated by pairs."""
    r, rest = x[..., :rotary_dim], x[..., rotary_dim:]
    if layout == "half":
        a, b = r[..., : rotary_dim // 2], r[..., rotary_dim // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def _plain_rotary(st):
    c, T = st["c"], st["c"]["T"]
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    row = st["row"].float().view(T, Hq + 2 * Hk, D)
    angle = st["pos"].double()[:, None, None] * st["freqs"].double()
    cos, sin = (torch.cos(angle) * st["magnitude"]).float(), (torch.sin(angle) * st["magnitude"]).float()
    q = _turn(row[:, :Hq], cos, sin, c["rotary_dim"], c["layout"])
    k = _turn(row[:, Hq:Hq + Hk], cos, sin, c["rotary_dim"], c["layout"])
    v = row[:, Hq + Hk:]
    if st["k_scale"] is not None:
        k = (k / st["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / st["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    # tokens without a slot write into a spare page behind the cache
    spare = st["pages"] * c["page"]
    slot = torch.where(st["slots"] < 0, spare, st["slots"])
    got = {"q": q.to(TYPES[c["dtype"]]).view(T, Hq * D)}
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


def _plain_attention(st):
    c = st["c"]
    B, Hq, Hk, D = c["B"], c["q_heads"], c["kv_heads"], c["head_dim"]
    table, n = st["table"].clamp(min=0).long(), st["lengths"][:, None]
    L = table.shape[1] * c["page"]
    t = torch.arange(L, device=DEV)
    seen = t < n
    if c["window"]:
        seen = seen & (t >= n - c["window"])
    k = st["k_cache"][table].transpose(1, 2).reshape(B, Hk, L, D).float()
    q = st["q"].float().view(B, Hk, Hq // Hk, D).transpose(2, 3).contiguous()
    s = (k @ q).transpose(2, 3) * st["scale"]
    del k
    if st["k_scale"] is not None:
        s = s * st["k_scale"][:, None, None]
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    v = st["v_cache"][table].transpose(1, 2).reshape(B, Hk, L, D).float()
    v = torch.where(seen[:, None, :, None], v, torch.zeros((), device=DEV))
    o = (p @ v) / torch.where(l == 0, torch.ones_like(l), l)
    if st["v_scale"] is not None:
        o = o * st["v_scale"][:, None, None]
    return {"out": o.reshape(B, Hq * D).to(TYPES[c["dtype"]]), "lse": (torch.log(l) + m).reshape(B, Hq)}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"product": _own_product, "rotary": _own_rotary, "attention": _own_attention}[op](state)
    return {"product": _plain_product, "rotary": _plain_rotary, "attention": _plain_attention}[op](state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        row = {"PQ2_0": K // 4, "Q2_0_G64": K // 4, "PTQ1_0": -(-K // 5), "Q1_0": K // 8}[c["fmt"]]
        b = N * (row + 2 * (K // _scale_group(c["fmt"]))) + 2 * M * K + 2 * M * N
        b += 2 * N * c["bias"] + 2 * M * N * (c["mul"] + c["residual"])
        return {"bytes": b, "flops": 2 * M * N * K}
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    kb = 1 if c["kv"] == "e4m3" else 2
    if c["op"] == "rotary":
        T = c["T"]
        b = T * (2 * D * (2 * Hq + 2 * Hk) + 2 * Hk * D * kb + 12) + 2 * c["rotary_dim"]
        return {"bytes": b, "flops": T * (Hq + Hk) * c["rotary_dim"] * 3}
    seen = [min(n, c["window"]) if c["window"] else n for n in _lengths(c)]
    b = 2 * sum(seen) * Hk * D * kb + 4 * c["B"] * Hq * D + 4 * c["B"] * (Hq + 1) + 4 * sum(-(-n // c["page"]) for n in seen)
    return {"bytes": b, "flops": 4 * sum(seen) * Hq * D}


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "product":
        x = st["x"].double()
        if c["rotate"]:
            i = torch.arange(128, device=DEV)
            both, parity = i[:, None] & i[None, :], torch.zeros((128, 128), dtype=torch.int64, device=DEV)
            for k in range(7):
                parity ^= (both >> k) & 1
            hadamard = (1 - 2 * parity).double() / math.sqrt(128.0)
            x = (x.view(c["M"], -1, 128) @ hadamard).reshape(c["M"], -1)
        grp = _scale_group(c["fmt"])
        y = torch.empty((c["M"], c["N"]), dtype=torch.float64, device=DEV)
        for r in range(0, c["N"], 4096):
            w = st["trits"][r: r + 4096].double() * st["scales"][r: r + 4096].double().repeat_interleave(grp, 1)
            y[:, r: r + 4096] = x @ w.t().contiguous()
        if c["bias"]:
            y += st["bias"].double()
        if c["act"] in ("relu", "relu2"):
            y = y.clamp(min=0) ** (2 if c["act"] == "relu2" else 1)
        elif c["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif c["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif c["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y))
        if c["mul"]:
            y *= st["mul"].double()
        if c["residual"]:
            y += st["residual"].double()
        return {"y": y}
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "rotary":
        T, R = c["T"], c["rotary_dim"]
        z = st["row"].double().view(T, Hq + 2 * Hk, D)
        turn = torch.polar(torch.full((T, 1, R // 2), st["magnitude"], dtype=torch.float64, device=DEV),
                           (st["pos"].double()[:, None] * st["freqs"].double())[:, None, :])
        first = torch.arange(R // 2, device=DEV) * (1 if c["layout"] == "half" else 2)
        second = first + (R // 2 if c["layout"] == "half" else 1)
        w = torch.complex(z[:, :Hq + Hk, first], z[:, :Hq + Hk, second]) * turn
        z[:, :Hq + Hk, first], z[:, :Hq + Hk, second] = w.real, w.imag
        got = {"q": z[:, :Hq].reshape(T, Hq * D)}
        kept = st["slots"] >= 0
        page, cell = st["slots"][kept] // c["page"], st["slots"][kept] % c["page"]
        for name, x in (("k", z[:, Hq:Hq + Hk]), ("v", z[:, Hq + Hk:])):
            if c["kv"] == "e4m3":
                x = torch.clamp(x / st[name + "_scale"].double()[:, None], -E4M3_MAX, E4M3_MAX)
            cache = st[name + "_cache_start"].double()
            cache[page, :, cell] = x[kept]
            got[name] = cache
        return got
    out = torch.zeros((c["B"], Hk, Hq // Hk, D), dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], Hk, Hq // Hk), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(c)):
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
            q = st["q"].double().view(c["B"], Hk, -1, D)[b, h]
            s = (q @ k.t().contiguous()) * st["scale"]
            lse[b, h] = torch.logsumexp(s, -1)
            out[b, h] = torch.exp(s - lse[b, h][:, None]) @ v
    return {"out": out.view(c["B"], Hq * D), "lse": lse.view(c["B"], Hq)}
