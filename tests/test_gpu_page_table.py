"""Block tables and slot maps against a plain walk over requests and tokens."""
from __future__ import annotations

import random

import pytest
import torch

import cache_reference as ref
from test_gpu_paged_attention import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(v, dev):  # noqa: F811
    return torch.tensor(v, dtype=torch.int32, device=dev)


def check(dev, cached, added, table, free, count, P, N, in_place=False):  # noqa: F811
    from memory_bound_moe_gb300 import PageTable, moe_page_table
    B, M = len(cached), len(table[0]) if table else 3
    t = i32(table, dev) if table else torch.empty((0, M), dtype=torch.int32, device=dev)
    c, fc = i32(cached, dev), i32([count], dev)
    junk = lambda n, dt=torch.int32: torch.full((n,), 12345, dtype=dt, device=dev)   # noqa: E731
    out = PageTable(c if in_place else junk(B), junk(B + 1), junk(N), junk(N, torch.int64), fc if in_place else junk(1), junk(1))
    free_t = i32(free, dev) if free else torch.empty(0, dtype=torch.int32, device=dev)
    got = moe_page_table(c, i32(added, dev), t, free_t, fc, P, N, out=out)
    rows = [list(r) for r in table]
    lengths, starts, positions, slots, left, refused = ref.page_table(cached, added, rows, free, count, P, N)
    assert got.lengths.tolist() == lengths
    assert got.starts.tolist() == [min(s, 2 ** 31 - 1) for s in starts]
    assert got.positions.tolist() == positions and got.slots.tolist() == slots
    assert got.free_count.tolist() == [left] and got.refused.tolist() == [refused]
    assert t.tolist() == rows
    return got


def random_step(rnd, B, P, M, most, N, enough):
    cached = [rnd.randint(0, max(0, M * P - most)) for _ in range(B)]
    added = [rnd.choice([0, 1, 1, 1, rnd.randint(0, most)]) for _ in range(B)]
    ids = list(range(B * M + 50))
    rnd.shuffle(ids)
    table = []
    for c in cached:
        have = -(-c // P)
        table.append([ids.pop() if j < have else -7 for j in range(M)])
    need = sum(-(-(c + a) // P) - -(-c // P) for c, a in zip(cached, added))
    count = need + rnd.randint(0, 9) if enough else rnd.randint(0, max(0, need - 1))
    free = ids[:min(len(ids), count + rnd.randint(0, 5))]
    return cached, added, table, free, min(count, len(free))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("enough", [True, False])
@pytest.mark.parametrize("B,P,M,most,N", [(1, 16, 4, 40, 64), (5, 1, 9, 4, 20), (16, 64, 20, 1, 16), (100, 16, 8, 30, 1000),
                                          (129, 8, 30, 200, 9000), (1025, 4, 6, 10, 3000), (3000, 32, 3, 3, 2900)])
def test_random_steps(dev, in_place, enough, B, P, M, most, N):  # noqa: F811
    rnd = random.Random(B * 7 + P + enough)
    for _ in range(3):
        check(dev, *random_step(rnd, B, P, M, most, N, enough), P, N, in_place)


def test_edges(dev):  # noqa: F811
    # no requests; no tokens; a prompt from nothing; exactly full pages; the last row's end
    check(dev, [], [], [], [3, 4], 2, 16, 5)
    check(dev, [0, 16], [0, 0], [[-1, -1], [9, -1]], [3, 4], 2, 16, 0)
    check(dev, [0], [64], [[-1] * 4], [5, 6, 7, 8], 4, 16, 64)
    check(dev, [16, 15, 32], [1, 1, 1], [[1, -1], [2, -1], [3, 4]], [5, 6], 2, 16, 3)   # the third passes its row
    # negative lengths, a negative and an excessive count, a negative page in use
    check(dev, [-4, 3], [2, -9], [[-1, -1], [0, -1]], [5, 6], 2, 16, 4)
    check(dev, [0, 3], [2, 1], [[-1, -1], [0, -1]], [5, 6], -3, 16, 4)
    check(dev, [0, 3], [2, 1], [[-1, -1], [-2, -1]], [5, 6], 100, 16, 4)
    check(dev, [0], [2], [[-1]], [], 0, 16, 4)
    # sums beyond 32 bits, tokens behind the capacity
    big = 2 ** 31 - 1
    check(dev, [big, 0, 4, 0], [big, big, 1, 1], [[-1, -1], [-1, -1], [8, -1], [-1, -1]], [5, 6], 2, 16, 10)
    check(dev, [0, 4, 0], [3, 8, 1], [[-1], [8], [-1]], [5, 6], 2, 16, 10)
    # pages run out at the second; requests without new pages go on, and so does none behind it that needs one
    check(dev, [0, 0, 3, 16], [16, 32, 1, 1], [[-1, -1], [-1, -1], [7, -1], [9, -1]], [5, 6], 2, 16, 50)


def test_pages_of_1024_and_the_most_requests(dev):  # noqa: F811
    rnd = random.Random(2)
    check(dev, *random_step(rnd, 50, 1024, 5, 3000, 60000, True), 1024, 60000)
    from memory_bound_moe_gb300 import MoeError
    check(dev, *random_step(rnd, 16384, 16, 2, 2, 20000, True), 16, 20000, in_place=True)
    with pytest.raises(MoeError):
        check(dev, [0] * 16385, [1] * 16385, [[-1]] * 16385, [1], 1, 16, 16385)


@pytest.mark.parametrize("B,P", [(1, 16), (40, 4), (1500, 16), (16384, 64)])
def test_release(dev, B, P):  # noqa: F811
    from memory_bound_moe_gb300 import moe_page_release
    rnd = random.Random(B)
    M = 5
    lengths = [rnd.choice([0, rnd.randint(1, M * P)]) for _ in range(B)]
    table = [[rnd.randint(0, 10 ** 6) for _ in range(M)] for _ in range(B)]
    finished = [rnd.choice([0, 0, 1, -3]) for _ in range(B)]
    free = [rnd.randint(0, 99) for _ in range(7)]
    back = [p for n, row, f in zip(lengths, table, finished) if f for p in row[:-(-n // P)]]
    for room in (len(back) + 3, len(back), max(0, len(back) - 2)):
        stack = i32(free + [-1] * room, dev)
        n, count, t = i32(lengths, dev), i32([len(free)], dev), i32(table, dev)
        moe_page_release(i32(finished, dev), t, n, stack, count, P)
        kept = (free + back)[:len(free) + room]
        assert count.tolist() == [len(kept)] and stack.tolist() == kept + [-1] * (len(free) + room - len(kept))
        assert n.tolist() == [0 if f else x for x, f in zip(lengths, finished)] and t.tolist() == table


def test_allocate_and_release_for_many_steps(dev):  # noqa: F811
    """Captured steps of a small serving loop: no page is ever held twice, none is lost."""
    from memory_bound_moe_gb300 import moe_page_release, moe_page_table
    rnd = random.Random(3)
    B, P, M, N, pages = 12, 4, 10, 40, 60
    lengths, added, finished = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(3))
    table = torch.full((B, M), -1, dtype=torch.int32, device=dev)
    free, count = torch.arange(pages, dtype=torch.int32, device=dev), i32([pages], dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe_page_release(finished, table, lengths, free, count, P)
        step = moe_page_table(lengths, added, table, free, count, P, N)
        lengths.copy_(step.lengths)
    refusals = 0
    for _ in range(100):
        finished.copy_(torch.tensor([int(rnd.random() < 0.08) for _ in range(B)]))
        added.copy_(torch.tensor([rnd.choice([0, 1, 1, rnd.randint(1, 9)]) for _ in range(B)]))
        graph.replay()
        held = [p for row, n in zip(table.tolist(), lengths.tolist()) for p in row[:-(-n // P)]]
        left = free.tolist()[:int(count)]
        assert sorted(held + left) == list(range(pages))
        used = [s for s in step.slots.tolist() if s >= 0]
        assert len(set(used)) == len(used) and {s // P for s in used} <= set(held)
        refusals += int(step.refused)
    assert refusals > 0
