"""Which table entries bgg_shared_attention goes by."""
import pytest

from test_gpu_shared_attention import Device, case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("pages", [1, 2, 5, 33])
@pytest.mark.parametrize("window", [0, 40])
def test_entries_of_the_shared_pages_name_other_pages(kv, pages, window):
    """The members after the first have pages of NaN in their entries of the
    shared pages, whose last may end inside a tile of 32 tokens."""
    c = case([(pages, [3, 9, 600, 0]), (1, [20, 30])], hq=4, hk=2, D=64, kv=kv, dtype="bf16" if kv == "bf16" else "f16",
             window=window, own_entries=False, seed=pages)
    nan = [torch.cat([x.float(), torch.full((1, *x.shape[1:]), float("nan"))]).to(x.dtype) for x in c["caches"]]
    c["caches"], c["pages"] = nan, c["pages"] + 1
    for b in (1, 2, 3):
        c["table"][b, :pages] = c["pages"] - 1
    c["table"][5, :1] = c["pages"] - 1
    d = Device(c)
    d.step()
    d.check()
