"""The longest prefix that a table can name: 2^31 - 16 tokens, whose last tile
ends at 2^31."""
import math

import pytest

import bit_gemv_gemm_amd as bgg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[2 ** 31 - 16, 2 ** 31 - 1], [2 ** 31 - 16, 5]])
def test_longest_prefix(lengths):
    """Every page is the same one, whose scores are 0, but for the last, of one
    token with a score of 60 and a value of its own: 2^31 e^-60 is 2^-55, so that
    token's value is the result of whoever sees it, and 60 its lse."""
    page, D, W = 16, 64, 0x7FFFFFFF // 16
    d = bgg.bgg_cache_describe("e4m3", 2, page, 1, D)
    k = torch.zeros((2, 1, page, D), dtype=torch.float32)
    v = torch.ones((2, 1, page, D), dtype=torch.float32)
    k[1, 0, 15, 0], v[1, 0, 15] = 60.0, 3.5
    k, v = (x.to(torch.float8_e4m3fn).cuda() for x in (k, v))
    q = torch.zeros((2, D), dtype=torch.float16, device="cuda")
    q[:, 0] = 1.0
    table = torch.zeros((2, W), dtype=torch.int32, device="cuda")
    table[0, -1] = 1  # (the second sequence's entries are not read)
    one = torch.ones(1, device="cuda")

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    out, lse = torch.zeros_like(q), torch.zeros(2, 1, device="cuda")
    ws = bgg.workspace(bgg.bgg_shared_attention_workspace_size(d, 1, 2))
    bgg.bgg_shared_attention(d, k, v, table, i32(lengths), i32([0, 2]), i32([W, W]), q, out, ws, scale=1.0, lse=lse, k_scale=one,
                             v_scale=one)
    torch.cuda.synchronize()
    for b, n in enumerate(lengths):
        long = n >= page * W
        assert (out[b].float() == (3.5 if long else 1.0)).all(), (b, out[b, :4])
        # test_gpu_attention's e + n 2^-23 + 2^-22 |lse| without the first two: the one product is exact, and one
        # probability, or five of 1, are the sum; the exponential of 2^-20 stays
        x = 60.0 if long else math.log(5)
        assert abs(lse[b].item() - x) <= 2.0 ** -20 + 2.0 ** -22 * x, (b, lse[b].item())


def test_infinite_values_at_the_end_of_the_longest_prefix():
    """The same table with an infinite and a NaN value of the last token."""
    page, D, W = 16, 64, 0x7FFFFFFF // 16
    d = bgg.bgg_cache_describe("f16", 2, page, 1, D)
    k, v = torch.zeros((2, 1, page, D)), torch.ones((2, 1, page, D))
    k[1, 0, 15, 0], v[1, 0, 15] = 60.0, 3.5
    v[1, 0, 15, 3], v[1, 0, 15, 5], v[1, 0, 14, 7] = float("inf"), float("nan"), -float("inf")
    k, v = k.half().cuda(), v.half().cuda()
    q = torch.zeros((2, D), dtype=torch.float16, device="cuda")
    q[:, 0] = 1.0
    table = torch.zeros((2, W), dtype=torch.int32, device="cuda")
    table[0, -1] = 1

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    out = torch.zeros_like(q)
    ws = bgg.workspace(bgg.bgg_shared_attention_workspace_size(d, 1, 2))
    bgg.bgg_shared_attention(d, k, v, table, i32([page * W] * 2), i32([0, 2]), i32([W, W]), q, out, ws, scale=1.0)
    torch.cuda.synchronize()
    want = torch.full((D,), 3.5)
    want[3], want[7] = float("inf"), -float("inf")
    for b in range(2):
        got = out[b].float().cpu()
        assert torch.isnan(got[5]) and torch.equal(torch.cat([got[:5], got[6:]]), torch.cat([want[:5], want[6:]])), (b, got[:9])
