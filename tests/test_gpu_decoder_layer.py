"""The operators of a decoder layer's decode step run together, as a program
would: grouped q|k|v product, rotary positions with the cache append, paged
attention, output product onto the residual stream, gated MLP -- for several
tokens of several sequences, eagerly and as one captured graph, against the
same layer in 64 bits.

Tolerance.  Each product is within 2e-3 of its row's largest value (the
products' own bar), and every 16-bit rounding adds 2^-11 of a value.  With
weights scaled so that each step keeps values of order one, six roundings and
four products in a row stay below 6 * 2^-11 + 4 * 2e-3 < 0.011 of the row's
largest value per step of the residual stream; 2e-2 covers the attention and
activation slopes (at most 1.13) between them."""
import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg
import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HQ, HK, D, HID, MLP, PAGE = 6, 2, 64, 384, 640, 16


class Matrix:
    def __init__(self, fmt, seed, N, K):
        T = synth.weights(fmt, seed, 0, N, K)
        S = (synth.scales_f16(seed, 0, N, K).astype(np.float64) * 2 / np.sqrt(K)).astype(np.float16)
        self.d = bgg.bgg_describe(fmt, N, K)
        self.packed = bgg.upload(bgg.bgg_pack_weights(self.d, T, S))
        self.host = (fmt, oracle.pack(fmt, T), S)
        self.N, self.K = N, K

    def exact(self, x):
        """W x' in 64 bits (x float64, model coordinates)."""
        fmt, packed, S = self.host
        W = oracle.unpack(fmt, packed, self.K).astype(np.float64) * np.repeat(S.astype(np.float64), 128, axis=1)
        H = np.array([[1.0]])
        while len(H) < 128:
            H = np.block([[H, H], [H, -H]])
        xr = (x.reshape(len(x), -1, 128) @ H / np.sqrt(128)).reshape(x.shape)
        return xr @ W.T


def layer(fmt):
    return dict(qkv=Matrix(fmt, 1, (HQ + 2 * HK) * D, HID), o=Matrix(fmt, 2, HID, HQ * D), gate=Matrix(fmt, 3, MLP, HID),
                up=Matrix(fmt, 4, MLP, HID), down=Matrix(fmt, 5, HID, MLP))


@pytest.mark.parametrize("fmt,kv", [("PQ2_0", "f16"), ("PTQ1_0", "f16")])
@pytest.mark.parametrize("B", [1, 3])
def test_decode_steps(fmt, kv, B):
    W, dev, steps = layer(fmt), "cuda", 40
    rng = np.random.default_rng(B)
    freqs, mag = bgg.bgg_rotary_frequencies(D, 10000.0, "parts", 4.0, trained_length=64.0)
    pages = B * 3 + 1
    cache = bgg.bgg_cache_describe(kv, pages, PAGE, HK, D)
    kc, vc = (torch.full((pages, HK, PAGE, D), float("nan"), dtype=torch.float16, device=dev) for _ in range(2))
    table = (torch.arange(B * 3).view(B, 3) + 1).flip(1).contiguous().int().to(dev)  # page 0 unused
    start = [0, 5, 7][:B]  # sequences of different ages
    ws = bgg.workspace(max(bgg.bgg_gemv_workspace_size(m.d, B) for m in W.values()))
    wsa = bgg.workspace(bgg.bgg_attention_workspace_size(cache, HQ, B))
    f16 = dict(dtype=torch.float16, device=dev)
    x, y = torch.zeros((B, HID), **f16), torch.zeros((B, HID), **f16)
    qkv, q, a = torch.zeros((B, W["qkv"].N), **f16), torch.zeros((B, HQ * D), **f16), torch.zeros((B, HQ * D), **f16)
    up, act = torch.zeros((B, MLP), **f16), torch.zeros((B, MLP), **f16)
    pos, slot = torch.zeros(B, dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int64, device=dev)
    n = torch.zeros(B, dtype=torch.int32, device=dev)
    fr = torch.from_numpy(freqs).to(dev)
    nq, nk = HQ * D, HK * D

    def step():
        rot = bgg.BGG_ROTATE_INPUT
        bgg.bgg_ternary_gemv(W["qkv"].d, W["qkv"].packed, x, qkv, B, rot, ws)
        bgg.bgg_rotary_append(cache, kc, vc, pos, slot, fr, q=qkv[:, :nq], q_out=q, k=qkv[:, nq:nq + nk],
                              v=qkv[:, nq + nk:], layout="half", magnitude=mag)
        bgg.bgg_paged_attention(cache, kc, vc, table, n, q, a, wsa, scale=D ** -0.5)
        bgg.bgg_ternary_gemv_epilogue(W["o"].d, W["o"].packed, a, y, B, rot, ws, residual=x)
        bgg.bgg_gemv_prepare(W["up"].d, y, B, rot, ws)
        bgg.bgg_gemv_run(W["up"].d, W["up"].packed, up, B, ws)
        bgg.bgg_gemv_run_epilogue(W["gate"].d, W["gate"].packed, act, B, ws, activation="silu", mul=up)
        bgg.bgg_ternary_gemv_epilogue(W["down"].d, W["down"].packed, act, y, B, rot, ws, residual=y)

    def exact(xs, ks, vs, p):
        z = W["qkv"].exact(xs)
        zq, zk, zv = z[:, :nq].reshape(B, HQ, D), z[:, nq:nq + nk].reshape(B, HK, D), z[:, nq + nk:].reshape(B, HK, D)
        ang = p[:, None, None] * freqs.astype(np.float64)

        def turn(v):
            u, w = v[..., :D // 2], v[..., D // 2:]
            return mag * np.concatenate([u * np.cos(ang) - w * np.sin(ang), u * np.sin(ang) + w * np.cos(ang)], -1)

        zq, zk = turn(zq), turn(zk)
        att = np.zeros((B, HQ, D))
        for b in range(B):
            ks[b].append(zk[b])
            vs[b].append(zv[b])
            for h in range(HQ):
                kk, vv = np.array(ks[b])[:, h // (HQ // HK)], np.array(vs[b])[:, h // (HQ // HK)]
                s = kk @ zq[b, h] / np.sqrt(D)
                e = np.exp(s - s.max())
                att[b, h] = e @ vv / e.sum()
        r = xs + W["o"].exact(att.reshape(B, -1))
        g = W["gate"].exact(r)
        return r + W["down"].exact(g / (1 + np.exp(-g)) * W["up"].exact(r))

    # a captured step and eager ones in turn
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    n.fill_(1)
    with torch.cuda.stream(side):
        step()  # (before the first token: writes slot 0, which page 0 leaves unused)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    ks, vs, ys = [[] for _ in range(B)], [[] for _ in range(B)], []
    # the sequences' first tokens, for those that are older
    for i in range(-max(start), steps):
        live = np.array([i >= -s for s in start])
        p = np.array([i + s if ok else 0 for s, ok in zip(start, live)])
        xs = rng.standard_normal((B, HID)).astype(np.float16)
        x.copy_(torch.from_numpy(xs))
        pos.copy_(torch.from_numpy(p.astype(np.int32)))
        tb = table.cpu().numpy()
        slot.copy_(torch.tensor([int(tb[b, p[b] // PAGE]) * PAGE + int(p[b] % PAGE) if live[b] else -1 for b in range(B)]))
        n.copy_(torch.from_numpy(np.where(live, p + 1, 0).astype(np.int32)))
        torch.cuda.synchronize()
        if i % 3 == 0:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        got = y.double().cpu().numpy()
        kb, vb = [list(v) for v in ks], [list(v) for v in vs]
        want = exact(xs.astype(np.float64), kb, vb, p.astype(np.float64))
        for b in range(B):
            if not live[b]:
                continue
            ks[b], vs[b] = kb[b], vb[b]
            e = np.max(np.abs(got[b] - want[b])) / np.max(np.abs(want[b]))
            assert e <= 2e-2, (i, b, e)
        ys.append(got)
    assert not ws[:16 << 20].any() and not wsa[:16384].any()
    assert not torch.isfinite(kc[0, :, 1:]).any()  # the unused page: only the step before the first token wrote there
