"""Paged attention where its ways of splitting the work meet: tables much wider
than the sequences, units around the number of blocks, random calls."""
from __future__ import annotations

import random

import pytest
import torch

from test_gpu_paged_attention import EDGES, KINDS, check, dev, make_cache, make_table, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def widened(table, P, tokens):
    """The same table with rows for `tokens` tokens; what lies behind the sequences is out of range."""
    wide = torch.full((table.shape[0], max(table.shape[1], -(-tokens // P))), -9, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 1), (6, 2), (9, 3), (32, 4), (64, 4), (20, 1)])
def test_wide_tables(dev, kind, D, Hq, Hkv):  # noqa: F811
    g = rng(dev, D + Hq)
    lengths = EDGES + [1000, 3000]
    table, pages = make_table(lengths, 16, dev, g)
    cache, k, v = make_cache(pages, 16, Hkv, D, kind, dev, g)
    q = torch.randn((len(lengths), Hq, D), generator=g, device=dev).to(torch.bfloat16)
    n = torch.tensor(lengths, dtype=torch.int32, device=dev)
    narrow = check(q, cache, k, v, table, n)
    wide = check(q, cache, k, v, widened(table, 16, 200000), n)
    for window in (1, 40, 999):
        check(q, cache, k, v, table, n, window=window)
    assert (narrow.float() - wide.float()).abs().max() <= 2.0 ** -6 * narrow.float().abs().max()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [1, 3, 32, 33, 34, 66, 67, 133, 134, 266, 267, 400])
def test_units_around_the_number_of_blocks(dev, kind, B):  # noqa: F811
    g = rng(dev, B)
    lengths = [(37 * i) % 230 for i in range(B)]
    table, pages = make_table(lengths, 8, dev, g)
    cache, k, v = make_cache(pages, 8, 1, 128, kind, dev, g)
    q = torch.randn((B, 5, 128), generator=g, device=dev).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(dev, seed):  # noqa: F811
    rnd = random.Random(seed)
    g = rng(dev, seed)
    Hkv, G, D, P = rnd.choice([1, 2, 3, 4, 5, 6, 8, 12]), rnd.choice([1, 2, 3, 5, 7, 8, 9, 12, 16, 18]), rnd.choice([64, 128, 256]), 2 ** rnd.randint(0, 8)
    kind, layout = rnd.choice(KINDS), rnd.choice(["token", "head", "joint"])
    B, top = rnd.choice([1, 2, 5, 17, 40]), rnd.choice([20, 300, 3000])
    lengths = [rnd.randint(0, top) for _ in range(B)]
    table, pages = make_table(lengths, P, dev, g)
    if rnd.random() < 0.5:
        table = widened(table, P, rnd.choice([1000, 20000, 300000]))
    cache, k, v = make_cache(pages, P, Hkv, D, kind, dev, g, layout)
    q = (rnd.choice([0.3, 1, 4]) * torch.randn((B, Hkv * G, D), generator=g, device=dev)).to(torch.bfloat16)
    window = rnd.choice([0, 0, 0, rnd.randint(1, top)])
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev), window=window)


def test_two_streams_with_their_own_workspaces(dev):  # noqa: F811
    """Calls in flight at once give what they give alone."""
    from memory_bound_moe_gb300 import moe_paged_attention, moe_paged_attention_workspace_size
    g = rng(dev, 3)
    jobs = []
    for B, top, kind in ((3, 30000, "bf16"), (40, 900, "e4m3"), (2, 200, "bf16")):
        lengths = [top - 7 * i for i in range(B)]
        table, pages = make_table(lengths, 16, dev, g)
        cache, k, v = make_cache(pages, 16, 4, 128, kind, dev, g)
        q = torch.randn((B, 32, 128), generator=g, device=dev).to(torch.bfloat16)
        n = torch.tensor(lengths, dtype=torch.int32, device=dev)
        ws = torch.empty(moe_paged_attention_workspace_size(B, 32, 4, 128), dtype=torch.uint8, device=dev)
        jobs.append((q, cache, table, n, ws, torch.empty_like(q), torch.cuda.Stream()))
    alone = [moe_paged_attention(q, c, t, n, workspace=ws).clone() for q, c, t, n, ws, _, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(30):
        for q, c, t, n, ws, out, s in jobs:
            moe_paged_attention(q, c, t, n, workspace=ws, out=out, stream=s)
    torch.cuda.synchronize()
    for (_, _, _, _, _, out, _), want in zip(jobs, alone):
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wide", [False, True])
def test_many_keys_that_are_not_numbers(dev, kind, wide):  # noqa: F811
    """A run of NaN keys, whoever reads it, makes its sequence's results NaN and no other's."""
    from memory_bound_moe_gb300 import moe_paged_attention
    g = rng(dev, 4)
    lengths = [700, 700, 700, 64, 20]
    table, pages = make_table(lengths, 16, dev, g)
    cache, k, v = make_cache(pages, 16, 1, 128, kind, dev, g)
    bits = k.view(torch.int16) if kind == "bf16" else k.view(torch.uint8)
    for b, (lo, hi) in enumerate(((0, 192), (512, 700), (0, 0), (0, 64), (0, 0))):
        for page in range(lo // 16, -(-hi // 16)):
            bits[int(table[b, page])] = 0x7fc0 if kind == "bf16" else 0x7f
    q = torch.randn((5, 4, 128), generator=g, device=dev).to(torch.bfloat16)
    if wide:
        table = widened(table, 16, 200000)
    out = moe_paged_attention(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device=dev))
    assert out[[0, 1, 3]].isnan().all() and out[[2, 4]].isfinite().all()


def test_values_of_very_different_size(dev):  # noqa: F811
    """Values near the largest bfloat16 at tokens whose weights vanish."""
    g = rng(dev, 6)
    lengths = [400, 33]
    table, pages = make_table(lengths, 16, dev, g)
    cache, k, v = make_cache(pages, 16, 1, 64, "bf16", dev, g)
    q = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=dev)
    q[..., 0] = 1.0
    # scores 0 for one token in eight, far below that for the others: weights of e^-60 to e^-400
    far = torch.arange(400, device=dev) % 8
    for b, n in enumerate(lengths):
        at = torch.arange(n, device=dev)
        page = table[b].long()[at // 16]
        k[page, at % 16, 0, 0] = -(far[:n] * 57 + (far[:n] > 0) * 3).to(torch.bfloat16)
        v[page, at % 16, 0, 1] = torch.where(far[:n] > 1, 3e38, 1.0).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev), scale=1.0)


def test_keys_and_values_laid_out_differently(dev):  # noqa: F811
    from memory_bound_moe_gb300 import KVCache
    g = rng(dev, 8)
    for P in (4, 32):
        lengths = [333, 0, 64, 5]
        table, pages = make_table(lengths, P, dev, g)
        _, k, _ = make_cache(pages, P, 4, 128, "bf16", dev, g, "token")
        _, _, v = make_cache(pages, P, 4, 128, "bf16", dev, g, "head")
        q = torch.randn((4, 8, 128), generator=g, device=dev).to(torch.bfloat16)
        n = torch.tensor(lengths, dtype=torch.int32, device=dev)
        check(q, KVCache(k, v), k, v, table, n)
        check(q, KVCache(k, v), k, v, widened(table, P, 200000), n)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1024, 8), (1024, 1024), (1023, 3)])
def test_the_most_heads(dev, kind, Hq, Hkv):  # noqa: F811
    g = rng(dev, Hkv)
    lengths = [90, 1, 0]
    table, pages = make_table(lengths, 16, dev, g)
    cache, k, v = make_cache(pages, 16, Hkv, 64, kind, dev, g)
    q = torch.randn((3, Hq, 64), generator=g, device=dev).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev))


def test_a_million_tokens_and_many_sequences(dev):  # noqa: F811
    g = rng(dev, 9)
    for lengths, P, kind in (([1000003, 5], 1024, "e4m3"), ([1000003, 70000], 16, "bf16"), ([i % 4 for i in range(5000)], 2, "bf16")):
        table, pages = make_table(lengths, P, dev, g)
        cache, k, v = make_cache(pages, P, 1, 64, kind, dev, g)
        q = (3 * torch.randn((len(lengths), 3, 64), generator=g, device=dev)).to(torch.bfloat16)
        check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev))


def test_two_graphs_that_share_a_workspace(dev):  # noqa: F811
    from memory_bound_moe_gb300 import moe_paged_attention, moe_paged_attention_workspace_size
    g = rng(dev, 10)
    ws = torch.empty(moe_paged_attention_workspace_size(9, 32, 4, 128), dtype=torch.uint8, device=dev)
    made = []
    for lengths, Hq, Hkv, wide in (([9000, 40, 3000], 32, 4, 200000), ([700] * 9, 16, 2, 0), ([20000], 8, 1, 0)):
        table, pages = make_table(lengths, 16, dev, g)
        table = widened(table, 16, wide) if wide else table
        cache, k, v = make_cache(pages, 16, Hkv, 128, "bf16", dev, g)
        q = torch.randn((len(lengths), Hq, 128), generator=g, device=dev).to(torch.bfloat16)
        n = torch.tensor(lengths, dtype=torch.int32, device=dev)
        want = check(q, cache, k, v, table, n, workspace=ws)
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe_paged_attention(q, cache, table, n, workspace=ws, out=out)
        made.append((graph, out, want, (cache, table, q, n)))   # a graph does not keep what it reads
    for _ in range(20):
        for graph, out, _, _ in made:
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _ in made:
        assert torch.equal(out, want)
