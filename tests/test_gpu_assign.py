"""cache_assign against the oracle's request-by-request assignment."""
import random

import pytest
import torch

import oracle
from _prompt import ints

pytestmark = pytest.mark.gpu


def state(rng, B, kv, new, page, count, width=None, ended=0.2, idle=0.2):
    """Requests with kv tokens at most, their pages in random order, and `count` free ones."""
    held = [rng.randint(0, kv) for _ in range(B)]
    add = [-1 if rng.random() < ended else 0 if rng.random() < idle else rng.randint(1, new) for _ in range(B)]
    need = [-(-n // page) for n in held]
    width = width or max([1] + [-(-(h + max(n, 0)) // page) for h, n in zip(held, add)])
    ids = list(range(sum(need) + count))
    rng.shuffle(ids)
    table = [[ids.pop() for _ in range(n)] + [-1] * (width - n) for n in need]
    free = ids + [-1] * (sum(need))
    return table, held, add, free


def run(ta, table, held, add, free, count, page, total, B, width, **kw):
    pages = torch.tensor(table, dtype=torch.int32).reshape(B, width).cuda()
    stack = ints(free)
    r = ta.cache_assign(pages, ints(held), ints(add), stack, ints([count]), page, total, **kw)
    return pages, stack, r


def compare(got, want, B, width):
    pages, stack, r = got
    table, free, kv, q, cu, pos, slots, count = want
    assert pages.cpu().tolist() == [list(x) for x in table] if B else True
    assert stack.cpu().tolist() == list(free)
    for name, x, y in (("kv_lens", r.kv_lens, kv), ("q_lens", r.q_lens, q), ("cu_seqlens", r.cu_seqlens, cu),
                       ("positions", r.positions, pos), ("slots", r.slots, slots), ("free_count", r.free_count, [count])):
        assert x.cpu().tolist() == list(y), name


@pytest.mark.parametrize("B,kv,new,page,spare,short", [
    (1, 0, 1, 1, 0, 0), (1, 30, 1, 16, 1, 0), (3, 50, 1, 7, 0, 0), (64, 300, 1, 16, 4, 0), (64, 100, 90, 8, 5, 0),
    (64, 100, 90, 8, 5, 0.5), (33, 40, 300, 64, 0, 0.3), (1023, 20, 9, 4, 3, 0), (1024, 20, 9, 4, 3, 0.6),
    (1025, 20, 9, 4, 3, 0), (2500, 12, 20, 5, 9, 0.7), (200, 64, 200, 24, 0, 0), (5, 3000, 4000, 32, 2, 0),
    (300, 500, 700, 8, 0, 0.8), (8192, 6, 5, 4, 2, 0), (8193, 6, 5, 4, 2, 0), (9001, 6, 5, 4, 2, 0.8),
])
@pytest.mark.parametrize("seed", [1, 2])
def test_against_the_oracle(gpu_lib, B, kv, new, page, spare, short, seed):
    ta = gpu_lib
    rng = random.Random(seed * 1000 + B)
    table, held, add, free = state(rng, B, kv, new, page, 0)
    width = len(table[0])
    want = sum(-(-(h + n) // page) - -(-h // page) for h, n in zip(held, add) if n > 0)
    count = int(want * (1 - short)) + spare
    used = sum(-(-h // page) for h in held)
    free = [used + i for i in range(count)] + [-1] * used
    total = sum(n for n in add if n > 0) + (3 if seed == 1 else 0)
    if short and seed == 2:
        total = total * 2 // 3
    ref = oracle.assign_pages(table, held, add, free, count, page, total)
    got = run(ta, table, held, add, free, count, page, total, B, width)
    assert ta.sync_status() == "TA_OK"
    compare(got, ref, B, width)
    # the inputs but the table and the stack are as they were: the same call gives the same
    pages, stack, r = got
    again = ta.cache_assign(pages, ints(held), ints(add), stack, ints([count]), page, total)
    compare((pages, stack, again), ref, B, width)


def test_steps_of_a_server(gpu_lib):
    """Steps one behind the other, each on the lengths and the stack that the one
    before left; no page is ever held twice."""
    ta = gpu_lib
    rng = random.Random(3)
    B, page, num, width = 40, 8, 90, 12
    table, kv, free, count = [[-1] * width for _ in range(B)], [0] * B, list(range(num)), num
    pages, lens, stack, n = torch.full((B, width), -1, dtype=torch.int32).cuda(), ints(kv), ints(free), ints([count])
    for step in range(30):
        add = []
        for b in range(B):
            room = page * width - kv[b]
            x = rng.random()
            add.append(-1 if kv[b] and x < 0.1 else 0 if x < 0.2 or room == 0 else
                       1 if kv[b] else rng.randint(1, min(room, 40)))
        total = 200
        table, free, kv, q, cu, pos, slots, count = oracle.assign_pages(table, kv, add, free, count, page, total)
        r = ta.cache_assign(pages, lens, ints(add), stack, n, page, total)
        compare((pages, stack, r), (table, free, kv, q, cu, pos, slots, count), B, width)
        lens, n = r.kv_lens.clone(), r.free_count.clone()
        held = [p for b in range(B) for p in table[b][:-(-kv[b] // page)]]
        assert len(set(held)) == len(held) and not set(held) & set(free[:count])
        assert len(held) + count == num
    assert ta.sync_status() == "TA_OK"


def test_no_requests_and_no_tokens(gpu_lib):
    ta = gpu_lib
    r = ta.cache_assign(torch.empty(0, 4, dtype=torch.int32, device="cuda"), ints([]), ints([]), ints([3, 1]), ints([2]), 4, 3)
    assert r.cu_seqlens.tolist() == [0] and r.slots.tolist() == [-1] * 3 and r.free_count.tolist() == [2]
    r = ta.cache_assign(ints([5]).view(1, 1), ints([2]), ints([0]), ints([]), ints([0]), 4, 0)
    assert r.kv_lens.tolist() == [2] and r.q_lens.tolist() == [0] and r.slots.numel() == 0
    assert ta.sync_status() == "TA_OK"


@pytest.mark.parametrize("kv,new,count,bad", [
    ([-1, 3], [1, 1], 4, 0), ([9, 3], [1, 1], 4, 0), ([3, 3], [6, 1], 4, 0), ([3, 3], [-2, 1], 4, 0),
    ([2 ** 31 - 1, 3], [2 ** 31 - 1, 1], 4, 0), ([9, 3], [-1, 1], 4, 0), ([3, 3], [1, 1], 5, None), ([3, 3], [1, 1], -1, None),
])
def test_what_cannot_be(gpu_lib, kv, new, count, bad):
    """Lengths past the page table (two pages of 4): the request stays idle and the
    others go on; a count that cannot be is 0.  Both are reported."""
    ta = gpu_lib
    pages = ints([0, 1, 2, 3]).view(2, 2)
    free = ints([4, 5, 6, 7])
    r = ta.cache_assign(pages, ints(kv), ints(new), free, ints([count]), 4, 8)
    assert ta.sync_status() == "TA_ERR_INDEX"
    if bad is not None:
        assert r.q_lens.tolist() == [0, 1] and r.kv_lens.tolist() == [kv[0], 4] and r.free_count.tolist() == [4]
        assert r.slots.tolist()[:2] == [2 * 4 + 3, -1]
    else:
        assert r.free_count.tolist() == [0] and r.q_lens.tolist() == [1, 1]


def test_page_ids_outside_the_cache(gpu_lib):
    ta = gpu_lib
    r = ta.cache_assign(ints([7, -5]).view(2, 1), ints([1, 1]), ints([1, 1]), ints([0, 1]), ints([2]), 4, 2)
    assert ta.sync_status() == "TA_ERR_INDEX" and r.slots.tolist() == [-1, -1] and r.positions.tolist() == [1, 1]
    # more pages come back than there are: the stack keeps what fits
    free = ints([0, 1])
    r = ta.cache_assign(ints([0, 1]).view(1, 2), ints([8]), ints([-1]), free, ints([1]), 4, 0)
    assert ta.sync_status() == "TA_ERR_INDEX" and r.free_count.tolist() == [2] and free.tolist() == [0, 0]


def test_replayed_from_a_graph_on_its_own_stream(gpu_lib):
    ta = gpu_lib
    rng = random.Random(4)
    B, page, total = 100, 8, 9000
    table, held, add, _ = state(rng, B, 60, 80, page, 0, width=20, ended=0.3)
    used = sum(-(-h // page) for h in held)
    free = [used + i for i in range(2000)] + [-1] * used
    pages, lens, new, stack, n = torch.tensor(table, dtype=torch.int32).cuda(), ints(held), ints(add), ints(free), ints([2000])
    keep = pages.clone(), stack.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ta.cache_assign(pages, lens, new, stack, n, page, total)
        with torch.cuda.graph(g, stream=side):
            r = ta.cache_assign(pages, lens, new, stack, n, page, total)
    torch.cuda.current_stream().wait_stream(side)
    pages.copy_(keep[0]), stack.copy_(keep[1])
    add = [n if n < 1 else rng.randint(1, 60) for n in add]
    new.copy_(ints(add))
    g.replay()
    torch.cuda.synchronize()
    compare((pages, stack, r), oracle.assign_pages(table, held, add, free, 2000, page, total), B, 20)
