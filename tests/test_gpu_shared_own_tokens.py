"""Own tokens of bgg_shared_attention in batches that one wave an item serves:
long sequences among short ones are cut for four times the items of workgroups
of four waves, and everything stays inside the workspace."""
import pytest

import bit_gemv_gemm_amd as bgg
from test_gpu_shared_attention import Device, case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GUARD = 1 << 16


def guarded(c, run):
    """run(Device) with guard bytes behind a workspace of exactly the stated size."""
    d = bgg.bgg_cache_describe(c["kv"], c["pages"], c["page"], c["hk"], c["D"])
    size = bgg.bgg_shared_attention_workspace_size(d, c["hq"], len(c["lengths"]))
    whole = torch.zeros(size + GUARD, dtype=torch.uint8, device="cuda")
    whole[size:] = 77
    run(Device(c, whole[:size]))
    torch.cuda.synchronize()
    assert (whole[size:] == 77).all() and not whole[:16384].any()


@pytest.mark.parametrize("dtype,kv,D,hq,hk", [("f16", "f16", 64, 16, 8), ("bf16", "bf16", 128, 8, 8), ("f16", "e4m3", 96, 24, 8),
                                              ("bf16", "bf16", 256, 4, 4)])
@pytest.mark.parametrize("long", [[3000] * 10, [40000], [600, 700, 20000, 1100, 513]])
def test_long_sequences_among_short_ones(dtype, kv, D, hq, hk, long):
    B = 1024 // hk + 2  # (at most 256 CUs)
    own = [(7 * b) % 45 for b in range(B)]
    at = [1 + (b * (B - 2)) // len(long) for b in range(len(long))]
    for b, n in zip(at, long):
        own[b] = n
    c = case([(4, own[:B // 3]), (9, own[B // 3:])], hq=hq, hk=hk, D=D, dtype=dtype, kv=kv, page=32, seed=D)
    rows = [(b, h) for b in at + [0, 2, B // 3, B - 1] for h in (0, hq // 2, hq - 1)]

    def run(d):
        d.step()
        d.check(rows)
        first = d.out.clone()
        d.out.fill_(float("nan"))
        d.step()
        torch.cuda.synchronize()
        assert torch.equal(first, d.out)

    guarded(c, run)


def test_every_sequence_cut():
    """As many parts as such a batch can have."""
    B, hk = 128, 8
    c = case([(1, [1100 + 7 * (b % 5) if b % 4 else 9 for b in range(B)])], hq=hk, hk=hk, D=64, kv="e4m3", seed=4)
    guarded(c, lambda d: (d.step(), d.check([(b, b % hk) for b in range(0, B, 3)])))
    c = case([(1, [5] * (B - 12) + [1300] * 12)], hq=hk, hk=hk, D=64, kv="e4m3", seed=5)
    guarded(c, lambda d: (d.step(), d.check([(b, b % hk) for b in [0, 3] + list(range(B - 13, B))])))


def test_workspace_grows_with_the_batch():
    size = bgg.bgg_shared_attention_workspace_size
    for args in (("f16", 10, 16, 8, 128), ("e4m3", 10, 64, 1, 64), ("bf16", 10, 16, 64, 256)):
        d = bgg.bgg_cache_describe(*args)
        sizes = [size(d, 2 * args[3], b) for b in (1, 2, 31, 32, 33, 127, 128, 129, 500, 1024, 1025, 4096)]
        assert sizes == sorted(sizes) and sizes[0] > bgg.bgg_attention_workspace_size(d, 2 * args[3], 1)
