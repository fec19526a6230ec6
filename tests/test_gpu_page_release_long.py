"""Pages given back by long rows: many pages a request, a stack that ends inside
a row, counts beyond 32 bits."""
from __future__ import annotations

import pytest
import torch

from test_gpu_paged_attention import dev, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room", [0, 1, 5000, None])
@pytest.mark.parametrize("P,lengths,finished", [
    (16, [131072], [1]),
    (1, [131072], [1]),
    (16, [40000, 0, 131071, 17, 65537, 131072], [1, 1, 1, 0, -2, 1]),
    (1, [131072, 5, 100000], [0, 1, 1]),
    (1024, [2 ** 20, 1025, 2 ** 20], [1, 1, 1])])
def test_long_rows(dev, P, lengths, finished, room):  # noqa: F811
    from memory_bound_moe_gb300 import moe_page_release
    g = rng(dev, len(lengths) + P)
    M = -(-max(lengths) // P) + 3
    table = torch.randint(0, 2 ** 31 - 1, (len(lengths), M), generator=g, device=dev).int()
    n, f = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (lengths, finished))
    back = torch.cat([table[b, :-(-x // P)] for b, x in enumerate(lengths) if finished[b]])
    room = back.numel() + 7 if room is None else room
    stack = torch.cat([torch.arange(9, device=dev), torch.full((room,), -1, device=dev)]).int()
    count, rows = torch.tensor([9], dtype=torch.int32, device=dev), table.clone()
    moe_page_release(f, table, n, stack, count, P)
    kept = back[:room]
    assert int(count) == 9 + kept.numel()
    assert torch.equal(stack[:9], torch.arange(9, device=dev).int()) and torch.equal(stack[9:9 + kept.numel()], kept)
    assert (stack[9 + kept.numel():] == -1).all() and torch.equal(table, rows)
    assert n.tolist() == [0 if x else y for x, y in zip(finished, lengths)]


def test_more_pages_than_32_bits_count(dev):  # noqa: F811
    """16384 requests of 131072 pages, 2^31 in all; the stack holds the first request's and a part of the second's."""
    from memory_bound_moe_gb300 import moe_page_release
    B, M = 16384, 131072
    table = torch.empty((B, M), dtype=torch.int32, device=dev)
    table[:2] = torch.arange(2 * M, dtype=torch.int32, device=dev).view(2, M)
    n, f = torch.full((B,), M, dtype=torch.int32, device=dev), torch.ones(B, dtype=torch.int32, device=dev)
    stack, count = torch.full((M + 1000,), -1, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    moe_page_release(f, table, n, stack, count, 1)
    assert int(count) == M + 1000 and torch.equal(stack, torch.arange(M + 1000, dtype=torch.int32, device=dev)) and (n == 0).all()
