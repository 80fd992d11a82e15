"""Samples of shared prompts decoded together, as a serving program would:
the page assignment of the prompts and of every step, q|k|v products, rotary
positions with several axes and the cache append, attention with shared
prefixes, output product onto the residual stream -- over many steps, some of
them replays of one captured step, with draft tokens given back in between,
against the same computation in 64 bits.

Tolerance: test_gpu_decoder_layer's for a step of a whole layer, of which this
is the first half (two products and four roundings of the values)."""
import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg
from test_gpu_decoder_layer import Matrix

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HQ, HK, D, HID, PAGE = 6, 2, 64, 384, 16
NQ, NK = HQ * D, HK * D
PROMPTS, MEMBERS = [37, 64], [3, 2]  # tokens of each prompt (the second ends with its page), its samples
SHARED = [n // PAGE for n in PROMPTS]
ALONE = 1  # a sequence of no group, behind them
B = sum(MEMBERS) + ALONE
T = B + 3  # rows of a step, three of them padding
SHIFT = [0, 3, 11]  # of the position on each axis
EMPTY = 300.0  # what no row may take over from the padding


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Program:
    def __init__(self, pages, fmt):
        self.qkv_w, self.o_w = Matrix(fmt, 1, NQ + 2 * NK, HID), Matrix(fmt, 2, HID, NQ)
        self.freqs, self.mag = bgg.bgg_rotary_frequencies(D, 10000.0, "none")
        self.axis = bgg.bgg_rotary_axes([12, 10, 10], "blocks")
        self.cache = bgg.bgg_cache_describe("f16", pages, PAGE, HK, D)
        f16 = dict(dtype=torch.float16, device="cuda")
        self.kc, self.vc = (torch.full((pages, HK, PAGE, D), float("nan"), **f16) for _ in range(2))
        self.free, self.count = i32(np.random.default_rng(3).permutation(pages).tolist()), i32([pages])
        self.fr, self.ax, self.shift = torch.from_numpy(self.freqs).cuda(), torch.from_numpy(self.axis).cuda(), i32(SHIFT)[:, None]
        self.ws = bgg.workspace(max(bgg.bgg_gemv_workspace_size(w.d, 16) for w in (self.qkv_w, self.o_w)))
        self.wsa = bgg.workspace(bgg.bgg_shared_attention_workspace_size(self.cache, HQ, B))

    def rows(self, n):
        """Buffers of a step of n rows."""
        f16 = dict(dtype=torch.float16, device="cuda")
        return dict(n=n, x=torch.zeros((n, HID), **f16), qkv=torch.zeros((n, NQ + 2 * NK), **f16), q=torch.zeros((n, NQ), **f16),
                    a=torch.zeros((B, NQ), **f16), y=torch.zeros((n, HID), **f16), pos=i32([0] * n),
                    pos3=torch.zeros((3, n), dtype=torch.int32, device="cuda"),
                    slots=torch.zeros(n, dtype=torch.int64, device="cuda"), past=i32([0] * 8), starts=i32([0] * 9))

    def assign(self, r, table, lengths, counts, shared=None):
        n = len(lengths)
        bgg.bgg_cache_assign(self.cache, lengths, counts, table, self.free, self.count, lengths, self.count, r["past"][:n],
                             r["starts"][:n + 1], r["pos"], r["slots"], shared_pages=shared)

    def fill(self, r):
        """Keys and values of the rows into the cache, queries into q."""
        for i in range(0, r["n"], 16):
            m = min(16, r["n"] - i)
            bgg.bgg_ternary_gemv(self.qkv_w.d, self.qkv_w.packed, r["x"][i:], r["qkv"][i:], m, bgg.BGG_ROTATE_INPUT, self.ws)
        torch.add(r["pos"], self.shift, out=r["pos3"])
        x = r["qkv"]
        bgg.bgg_rotary_append_axes(self.cache, self.kc, self.vc, r["pos3"], self.ax, r["slots"], self.fr, q=x[:, :NQ],
                                   q_out=r["q"], k=x[:, NQ:NQ + NK], v=x[:, NQ + NK:], layout="half", magnitude=self.mag)

    def attend(self, r, table, lengths, starts, shared):
        bgg.bgg_shared_attention(self.cache, self.kc, self.vc, table, lengths, starts, shared, r["q"][:B], r["a"], self.wsa,
                                 scale=D ** -0.5)
        bgg.bgg_ternary_gemv_epilogue(self.o_w.d, self.o_w.packed, r["a"], r["y"][:B], B, bgg.BGG_ROTATE_INPUT,
                                      self.ws, residual=r["x"][:B])

    def exact_kv(self, x, p):
        """q, k, v of rows x at positions p."""
        z = self.qkv_w.exact(x)
        ang = (p[:, None] + np.array(SHIFT)[self.axis]) * self.freqs.astype(np.float64)

        def turn(v):
            u, w = v[..., :D // 2], v[..., D // 2:]
            c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
            return self.mag * np.concatenate([u * c - w * s, u * s + w * c], -1)

        n = len(x)
        return (turn(z[:, :NQ].reshape(n, HQ, D)), turn(z[:, NQ:NQ + NK].reshape(n, HK, D)), z[:, NQ + NK:].reshape(n, HK, D))


@pytest.mark.parametrize("fmt", ["PQ2_0", "PTQ1_0"])
def test_samples_of_shared_prompts(fmt):
    rng = np.random.default_rng(1)
    prog = Program(pages=64, fmt=fmt)

    # the prompts, one sequence each
    total = sum(PROMPTS)
    r = prog.rows(total)
    prompt_table, prompt_len = i32([[-1] * 5] * 2), i32([0, 0])
    xs = rng.standard_normal((total, HID)).astype(np.float16)
    r["x"].copy_(torch.from_numpy(xs))
    prog.assign(r, prompt_table, prompt_len, i32(PROMPTS))
    prog.fill(r)
    assert prompt_len.tolist() == PROMPTS and r["starts"][:3].tolist() == [0, PROMPTS[0], total]
    prompt_x = np.split(xs.astype(np.float64), [PROMPTS[0]])
    # what does not fill a page is given back, to be each sample's own
    prog.assign(r, prompt_table, prompt_len, i32([s * PAGE - n for s, n in zip(SHARED, PROMPTS)]))
    assert prompt_len.tolist() == [s * PAGE for s in SHARED] and prog.count.item() == 64 - sum(SHARED)

    # the samples
    group_of = [g for g, m in enumerate(MEMBERS) for _ in range(m)] + [None] * ALONE
    starts = i32([0] + np.cumsum(MEMBERS).tolist())
    shared = i32([SHARED[g] if g is not None else 0 for g in group_of])
    table = i32([[-1] * 12] * B)
    for b, g in enumerate(group_of):
        if g is not None:
            table[b, :SHARED[g]] = prompt_table[g, :SHARED[g]]
    lengths = shared * PAGE
    ks, vs = [], []
    for g in group_of:
        k, v = [], []
        if g is not None:
            _, k, v = prog.exact_kv(prompt_x[g][:SHARED[g] * PAGE], np.arange(SHARED[g] * PAGE))
        ks.append(list(k)), vs.append(list(v))
    # the rest of the prompt, for every sample (of the one alone, five tokens of its own)
    tails = [prompt_x[g][SHARED[g] * PAGE:] if g is not None else rng.standard_normal((5, HID)).astype(np.float16).astype(np.float64)
             for g in group_of]
    r = prog.rows(sum(map(len, tails)) + 2)
    r["x"][:-2] = torch.from_numpy(np.concatenate(tails).astype(np.float16))
    prog.assign(r, table, lengths, i32([len(t) for t in tails]), shared)
    prog.fill(r)
    for b, t in enumerate(tails):
        if len(t):
            _, k, v = prog.exact_kv(t, len(ks[b]) + np.arange(len(t)))
            ks[b] += list(k)
            vs[b] += list(v)
    assert lengths.tolist() == [len(k) for k in ks] and r["slots"][-2:].tolist() == [-1, -1]

    # a token of each sample per step
    r = prog.rows(T)
    one = i32([1] * B)

    def step():
        prog.assign(r, table, lengths, one, shared)
        prog.fill(r)
        prog.attend(r, table, lengths, starts, shared)

    def check(xs, i):
        want = np.zeros((B, HID))
        att = np.zeros((B, HQ, D))
        q, k, v = prog.exact_kv(xs, np.array([len(x) for x in ks]))
        for b in range(B):
            ks[b].append(k[b])
            vs[b].append(v[b])
            kk, vv = np.array(ks[b]), np.array(vs[b])
            for h in range(HQ):
                s = kk[:, h // (HQ // HK)] @ q[b, h] / np.sqrt(D)
                e = np.exp(s - s.max())
                att[b, h] = e @ vv[:, h // (HQ // HK)] / e.sum()
        want = xs + prog.o_w.exact(att.reshape(B, -1))
        got = r["y"].double().cpu().numpy()
        assert lengths.tolist() == [len(x) for x in ks], i
        assert r["slots"][B:].tolist() == [-1] * (T - B)
        for b in range(B):
            e = np.max(np.abs(got[b] - want[b])) / np.max(np.abs(want[b]))
            assert e <= 2e-2, (i, b, e)
        assert (got[B:] == EMPTY).all(), "rows behind the last sequence"

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    for i in range(45):
        xs = rng.standard_normal((B, HID)).astype(np.float16)
        r["x"].zero_()
        r["x"][:B] = torch.from_numpy(xs)
        r["y"].fill_(EMPTY)
        torch.cuda.synchronize()
        if i == 1:
            with torch.cuda.stream(side):
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.graph(graph, stream=side):
                    step()
            torch.cuda.synchronize()
        if i == 0 or i % 5 == 4:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        check(xs.astype(np.float64), i)
        if i % 7 == 6:  # some of the last tokens are given back, over the ends of pages and down to the shared ones
            back = [min(n, len(x) - int(s) * PAGE) for n, x, s in zip([3, 40, 1, 0, 17, 2], ks, shared.tolist())]
            prog.assign(prog.rows(0), table, lengths, i32([-3, -40, -1, 0, -17, -2]), shared)
            for b, n in enumerate(back):
                del ks[b][len(ks[b]) - n:], vs[b][len(vs[b]) - n:]
            assert lengths.tolist() == [len(x) for x in ks]
            held = [-(-len(x) // PAGE) - int(s) for x, s in zip(ks, shared.tolist())]
            assert prog.count.item() == 64 - sum(SHARED) - sum(held), "every page is held once or free"
    assert not prog.ws[:16 << 20].any() and not prog.wsa[:16384].any()
