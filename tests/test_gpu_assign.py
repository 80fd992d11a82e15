"""Page tables and slots built from the lengths of a batch's sequences,
against a stack of free pages kept one sequence after the other on the host.
Whole numbers: everything is compared for equality, the untouched parts of
the table, of the stack and of what lies around the outputs included."""
import random

import pytest

import bit_gemv_gemm_amd as bgg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
MIN = -(1 << 31)


def held(n, ps):
    return -(-n // ps)


def step(ps, W, T, pages, capacity, lengths, counts, table, stack, count, shared=None):
    """The definition, on lists; table and stack are changed in place."""
    B = len(lengths)
    n = [min(max(v, 0), W * ps) for v in lengths]
    low = [min(max(v, 0), W) * ps for v in shared] if shared is not None else [0] * B
    top = min(max(count, 0), capacity)
    past = [min(n[b], max(n[b] + counts[b], low[b])) if counts[b] < 0 else n[b] for b in range(B)]
    for b in reversed(range(B)):
        for p in reversed(range(held(past[b], ps), held(n[b], ps))):
            if 0 <= table[b][p] < pages and top < capacity:
                stack[top] = table[b][p]
                top += 1
    after, starts, positions, slots, row, closed = list(past), [0], [0] * T, [-1] * T, 0, False
    for b in range(B):
        c, first = max(counts[b], 0), row
        row += c
        starts.append(min(row, T))
        if row > T or past[b] + c > W * ps:
            continue
        wanted = range(held(past[b], ps), held(past[b] + c, ps))
        if len(wanted) and (closed or len(wanted) > top):
            closed = True
            continue
        for p in wanted:
            top -= 1
            table[b][p] = stack[top]
        after[b] = past[b] + c
        for i in range(c):
            at = past[b] + i
            page = table[b][at // ps]
            positions[first + i] = at
            slots[first + i] = page * ps + at % ps if 0 <= page < pages else -1
    return dict(lengths_out=after, free_count_out=[top], past=past, starts=starts, positions=positions, slots=slots)


GUARD = 7


class Buffers:
    """Device arrays with guard values around them."""

    def __init__(self, B, T):
        self.whole = {}
        for name, n, dt in (("lengths_out", B, torch.int32), ("free_count_out", 1, torch.int32), ("past", B, torch.int32),
                            ("starts", B + 1, torch.int32), ("positions", T, torch.int32), ("slots", T, torch.int64)):
            w = torch.full((n + 2 * GUARD,), 12345, dtype=dt, device=DEV)
            self.whole[name] = w
            setattr(self, name, w[GUARD:GUARD + n])

    def check(self, want):
        for name, w in self.whole.items():
            got = w.tolist()
            assert got[:GUARD] == got[len(got) - GUARD:] == [12345] * GUARD, name
            assert got[GUARD:-GUARD] == want[name], name


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def run_case(seed, B, ps, W, T, mode, short=0, extra_stride=0, shared=None, capacity_cut=0):
    r = random.Random(seed)
    lengths, counts = [], []
    left = T
    for b in range(B):
        n = r.choice([0, 1, ps - 1, ps, ps + 1, r.randint(0, W * ps), r.randint(0, W * ps)])
        n = min(n, W * ps)
        if shared is not None:
            n = max(n, min(shared[b], W) * ps)
        if mode == "one":
            c = 1
        elif mode == "cut":
            c = r.choice([-1, -n, MIN, 0, -r.randint(0, 2 * ps), 1])
        else:
            c = r.choice([0, 0, 1, 1, 2, ps, r.randint(0, 3 * ps), max(0, W * ps - n), W * ps - n + 1, -r.randint(0, 40), MIN])
            if c > left and r.random() < 0.9:
                c = r.randint(0, left)
        left -= max(0, min(c, left))
        lengths.append(n)
        counts.append(c)
    if mode == "mixed" and B > 3:
        lengths[1], lengths[2] = -5, W * ps + 3  # cut to 0 .. W ps
    need = sum(max(0, held(n + c, ps) - held(n, ps)) for n, c in zip(lengths, counts) if c > 0)
    pages = B * W + need + 5
    order = list(range(pages))
    r.shuffle(order)
    table = [[-1] * W for _ in range(B)]
    at = 0
    for b in range(B):
        for p in range(min(held(max(lengths[b], 0), ps), W)):
            table[b][p] = order[at] if r.random() < 0.95 else r.choice([-1, pages, MIN, 2**31 - 1])
            at += 1
    free = order[at:at + max(1, need - short)] if need else order[at:at + 3]
    capacity = max(1, pages - capacity_cut)
    stack = free[:capacity] + [-7] * (capacity - len(free))
    if len(free) > 2 and mode == "mixed":
        stack[0] = pages + 1  # a page number that lies outside: it gives no slot
    count = min(len(free), capacity)
    stride = W + extra_stride
    whole = torch.full((B, stride), -99, dtype=torch.int32, device=DEV)
    dt = whole[:, :W]
    if B:
        dt.copy_(i32(table))
    dstack = i32(stack)
    buf = Buffers(B, T)
    cache = bgg.bgg_cache_describe("f16", pages, ps, 1, 64)
    bgg.bgg_cache_assign(cache, i32(lengths), i32(counts), dt, dstack, i32([count]), buf.lengths_out, buf.free_count_out,
                         buf.past, buf.starts, buf.positions, buf.slots,
                         shared_pages=None if shared is None else i32(shared))
    torch.cuda.synchronize()
    want = step(ps, W, T, pages, capacity, lengths, counts, table, stack, count, shared)
    buf.check(want)
    assert dt.tolist() == table
    assert dstack.tolist() == stack
    if extra_stride and B:
        assert (whole[:, W:] == -99).all()
    return want


@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 255, 256, 257, 1000, 1025, 4096])
@pytest.mark.parametrize("mode", ["one", "cut", "mixed"])
def test_batches(B, mode):
    run_case(B, B, 16, 9, B if mode == "one" else 3 * B + 17, mode)


@pytest.mark.parametrize("ps,W", [(16, 1), (32, 40), (64, 3), (256, 2), (65536, 2), (1024, 300)])
@pytest.mark.parametrize("T", [1, 64, 4095, 4096, 4097, 8200, 30011])
def test_rows_around_the_own_launch(ps, W, T):
    run_case(T + ps, 37, ps, W, T, "mixed")


@pytest.mark.parametrize("B", [37, 256])
@pytest.mark.parametrize("T", [1023, 1024, 1025, 2047, 2049])
def test_rows_around_the_own_launch_of_small_batches(B, T):
    run_case(T + B, B, 16, 60, T, "mixed")


@pytest.mark.parametrize("B", [257, 1023, 1024, 1025, 4096])
@pytest.mark.parametrize("T", [4096, 4097, 9001])
def test_rows_of_large_batches(B, T):
    run_case(T + B, B, 16, 8, T, "mixed", extra_stride=1)


@pytest.mark.parametrize("B", [5, 600, 3000])
def test_one_long_sequence_among_unused_ones(B):
    """Its rows are those of many workgroups, none of which hold its first."""
    ps, W, T, at, n, c = 32, 700, 20000, B // 2, 45, 19990
    counts = [c if b == at else 0 for b in range(B)]
    lengths = [n if b == at else 0 for b in range(B)]
    pages = W + 3
    table, stack = [[-1] * W for _ in range(B)], list(range(pages - 2))
    table[at][:2] = [pages - 1, pages - 2]
    dt, dstack, buf = i32(table), i32(stack), Buffers(B, T)
    cache = bgg.bgg_cache_describe("f16", pages, ps, 1, 64)
    bgg.bgg_cache_assign(cache, i32(lengths), i32(counts), dt, dstack, i32([len(stack)]), buf.lengths_out, buf.free_count_out,
                         buf.past, buf.starts, buf.positions, buf.slots)
    torch.cuda.synchronize()
    buf.check(step(ps, W, T, pages, len(stack), lengths, counts, table, stack, len(stack)))
    assert dt.tolist() == table and dstack.tolist() == stack


@pytest.mark.parametrize("T", [600, 20000])
@pytest.mark.parametrize("B", [9, 300])
@pytest.mark.parametrize("short", [1, 2, 5, 100])
def test_too_few_pages(B, T, short):
    want = run_case(7 * B + short, B, 16, 30, T, "mixed", short=short)
    assert want["free_count_out"][0] >= 0


def test_more_pages_back_than_room():
    run_case(3, 40, 16, 12, 100, "cut", capacity_cut=400)


def test_many_pages_back():
    # 2000 entries of each of 5 sequences: several rounds of the workgroup
    run_case(11, 5, 16, 2000, 10, "cut", extra_stride=3)


@pytest.mark.parametrize("T", [50, 9000])
def test_shared_pages_stay(T):
    r = random.Random(5)
    run_case(8, 50, 32, 20, T, "mixed", shared=[r.choice([0, 1, 7, 20, 25, -3]) for _ in range(50)], extra_stride=5)


@pytest.mark.parametrize("T", [0, 5, 5000])
def test_no_sequences_and_no_rows(T):
    run_case(1, 0, 16, 4, T, "one")
    run_case(2, 6, 16, 4, 0, "cut")
    run_case(2, 6, 16, 4, 0, "mixed")


@pytest.mark.parametrize("T", [10, 6000])
def test_largest_counts(T):
    # counts whose sum passes 32 bits are not served; the sequences among them that fit the rows are
    ps, W = 16, 1 << 20
    counts = [2, 2**31 - 1, 2**31 - 1, 3, 2**31 - 1, 0, MIN]
    lengths = [0, 5, W * ps, 0, 2**31 - 1, 17, 2**31 - 1]
    table = torch.full((7, W), -1, dtype=torch.int32, device=DEV)
    buf = Buffers(7, T)
    stack = i32([3, 1, 2, 0])
    cache = bgg.bgg_cache_describe("f16", 4, ps, 1, 64)
    bgg.bgg_cache_assign(cache, i32(lengths), i32(counts), table, stack, i32([4]), buf.lengths_out, buf.free_count_out,
                         buf.past, buf.starts, buf.positions, buf.slots)
    torch.cuda.synchronize()
    buf.check(dict(lengths_out=[2, 5, W * ps, 0, W * ps, 17, 0], free_count_out=[3], past=[0, 5, W * ps, 0, W * ps, 17, 0],
                   starts=[0, 2, T, T, T, T, T, T], positions=[0, 1] + [0] * (T - 2), slots=[0, 1] + [-1] * (T - 2)))


def test_a_step_given_back_leaves_the_stack_as_it_was():
    B, ps, W, T = 33, 16, 8, 400
    r = random.Random(9)
    pages = B * W
    order = list(range(pages))
    r.shuffle(order)
    stack, count, lengths = i32(order), i32([pages]), i32([0] * B)
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    cache = bgg.bgg_cache_describe("f16", pages, ps, 1, 64)
    past, starts = i32([0] * B), i32([0] * (B + 1))
    pos, slots = torch.zeros(T, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int64, device=DEV)
    new = [r.randint(0, 12) for _ in range(B)]

    def go(c):
        bgg.bgg_cache_assign(cache, lengths, i32(c), table, stack, count, lengths, count, past, starts, pos, slots)

    go(new)
    before = (stack.clone(), count.clone(), lengths.clone())
    go([20] * B)  # draft tokens, all rejected
    go([-20 if n else 0 for n in (lengths - before[2]).tolist()])
    torch.cuda.synchronize()
    assert torch.equal(lengths, before[2]) and torch.equal(count, before[1])
    assert torch.equal(stack[:int(count)], before[0][:int(count)])


def test_captured_steps_in_place():
    """Lengths, stack and table change in place over many steps, some of them
    replays of one captured step and some eager, against the host's stack."""
    B, ps, W, T = 21, 16, 6, 64
    r = random.Random(4)
    pages = 60  # too few for all
    order = list(range(pages))
    r.shuffle(order)
    stack, table, lengths, count = list(order), [[-1] * W for _ in range(B)], [0] * B, pages
    dstack, dtable, dlen, dcount = i32(stack), i32(table), i32(lengths), i32([count])
    dc = i32([0] * B)
    past, starts = i32([0] * B), i32([0] * (B + 1))
    pos, slots = torch.zeros(T, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int64, device=DEV)
    cache = bgg.bgg_cache_describe("bf16", pages, ps, 1, 64)

    def go():
        bgg.bgg_cache_assign(cache, dlen, dc, dtable, dstack, dcount, dlen, dcount, past, starts, pos, slots)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        go()  # nothing new: changes nothing
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            go()
    torch.cuda.synchronize()
    for i in range(60):
        counts = [r.choice([0, 1, 1, 1, 2, 5, 17, -1, -3, MIN if r.random() < 0.2 else 1]) for _ in range(B)]
        dc.copy_(i32(counts))
        torch.cuda.synchronize()
        graph.replay() if i % 3 else go()
        torch.cuda.synchronize()
        want = step(ps, W, T, pages, pages, lengths, counts, table, stack, count)
        lengths, count = want["lengths_out"], want["free_count_out"][0]
        assert dlen.tolist() == lengths and dcount.item() == count, i
        assert dtable.tolist() == table and dstack.tolist() == stack, i
        assert past.tolist() == want["past"] and starts.tolist() == want["starts"], i
        assert pos.tolist() == want["positions"] and slots.tolist() == want["slots"], i
        # no page has two owners
        held_pages = [p for b in range(B) for p in table[b][:held(lengths[b], ps)]]
        assert sorted(held_pages + stack[:count]) == list(range(pages)), i


def test_on_another_stream():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_case(77, 300, 16, 9, 6000, "mixed")


def test_refusals_of_the_binding():
    cache = bgg.bgg_cache_describe("f16", 4, 16, 1, 64)
    good = dict(lengths=i32([0, 0]), counts=i32([1, 1]), page_table=i32([[-1], [-1]]), free_pages=i32([0, 1]),
                free_count=i32([2]), lengths_out=i32([0, 0]), free_count_out=i32([0]), past=i32([0, 0]),
                starts=i32([0, 0, 0]), positions=i32([0, 0]), slots=torch.zeros(2, dtype=torch.int64, device=DEV))
    bgg.bgg_cache_assign(cache, **good)
    torch.cuda.synchronize()
    assert good["slots"].tolist() == [16, 0]
    for name, bad in [("lengths", good["lengths"].cpu()), ("counts", i32([1])), ("counts", good["counts"].long()),
                      ("page_table", i32([[-1]])), ("page_table", i32([-1, -1])), ("free_pages", None),
                      ("free_count", i32([])), ("starts", i32([0, 0])), ("slots", good["slots"].int()),
                      ("slots", good["slots"][:1]), ("past", None), ("positions", None), ("lengths_out", i32([0])),
                      ("page_table", torch.zeros((2, 2), dtype=torch.int32, device=DEV).t()[:, :1].expand(2, 3))]:
        with pytest.raises((ValueError, TypeError)):
            bgg.bgg_cache_assign(cache, **dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        bgg.bgg_cache_assign(cache, **good, shared_pages=i32([0]))
