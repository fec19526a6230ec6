"""Attention of one token per sequence over a paged cache, against float64."""
from __future__ import annotations

import math

import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu
KINDS = ("bf16", "e4m3")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_moe_gb300 import build
    build.build()
    return torch.device("cuda:0")


def make_cache(pages, P, Hkv, D, kind, dev, gen, layout="token"):
    """(KVCache, k, v): unit values, E4M3 ones at scales that are no powers of two."""
    from memory_bound_moe_gb300 import KVCache

    def side(std):
        shape = (pages, Hkv, P, D) if layout == "head" else (pages, P, 2, Hkv, D) if layout == "joint" else (pages, P, Hkv, D)
        t = torch.randn(shape, generator=gen, device=dev) * std
        t = t.to(torch.bfloat16) if kind == "bf16" else t.clamp(-448, 448).to(torch.float8_e4m3fn)
        return t.transpose(1, 2) if layout == "head" else t[:, :, 0] if layout == "joint" else t

    if kind == "bf16":
        k, v = side(1.0), side(1.0)
        return KVCache(k, v), k, v
    k, v = side(40.0), side(60.0)
    return KVCache(k, v, 0.021, 0.017), k, v


def make_table(lengths, P, dev, gen, spare=2):
    """(block table, pages): shuffled pages; entries behind a sequence are far outside the cache."""
    need = [-(-n // P) for n in lengths]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=gen, device=dev).int()
    table = torch.full((len(lengths), max(need + [1])), 2 ** 31 - 1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pages


def check(q, cache, k, v, table, lengths, scale=None, window=0, **kw):
    from memory_bound_moe_gb300 import moe_paged_attention
    B, Hq, D = q.shape
    lse = torch.full((B, Hq), 7.0, device=q.device)
    out = moe_paged_attention(q, cache, table, lengths, scale=scale, window=window, lse=lse, **kw)
    again = moe_paged_attention(q, cache, table, lengths, scale=scale, window=window, **kw)
    want, want_lse, tol, ltol = ref.attention(q, k, v, table, lengths, D ** -0.5 if scale is None else scale, window,
                                              cache.k_scale, cache.v_scale)
    off = (out.double() - want).abs()
    assert out.isfinite().all()
    assert (off <= tol).all(), f"out: {float((off / tol.clamp_min(1e-300)).max()):.3g} of the bound"
    empty = want_lse == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    loff = (lse.double() - want_lse)[~empty].abs()
    assert (loff <= ltol[~empty]).all(), f"lse: {float((loff / ltol[~empty]).max()):.3g} of the bound"
    assert torch.equal(out, again)
    return out


def rng(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (8, 8), (16, 1), (32, 4)])
def test_heads_and_edge_lengths(dev, kind, D, Hq, Hkv):
    g = rng(dev, D + Hq)
    table, pages = make_table(EDGES, 16, dev, g)
    cache, k, v = make_cache(pages, 16, Hkv, D, kind, dev, g)
    q = (2 * torch.randn((len(EDGES), Hq, D), generator=g, device=dev)).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(EDGES, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["token", "head", "joint"])
@pytest.mark.parametrize("P", [1, 2, 4, 8, 32, 128, 1024])
def test_page_sizes_and_layouts(dev, kind, layout, P):
    g = rng(dev, P)
    lengths = [P, P + 1, 0, max(P - 1, 1), 3 * P + 7, 500]
    table, pages = make_table(lengths, P, dev, g)
    cache, k, v = make_cache(pages, P, 3, 128, kind, dev, g, layout)
    q = torch.randn((len(lengths), 12, 128), generator=g, device=dev).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(17, 1), (40, 1), (128, 2)])
def test_groups_of_more_than_16_heads(dev, kind, Hq, Hkv):
    g = rng(dev, Hq)
    lengths = [3000, 1, 0, 777]
    table, pages = make_table(lengths, 32, dev, g)
    cache, k, v = make_cache(pages, 32, Hkv, 64, kind, dev, g)
    q = torch.randn((4, Hq, 64), generator=g, device=dev).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 15, 16, 17, 64, 100, 1000, 5000])
def test_windows(dev, kind, window):
    g = rng(dev, window)
    lengths = [0, 1, 16, 17, 99, 100, 101, 1023, 4999, 2047]
    table, pages = make_table(lengths, 16, dev, g)
    cache, k, v = make_cache(pages, 16, 2, 128, kind, dev, g)
    q = torch.randn((len(lengths), 16, 128), generator=g, device=dev).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev), window=window)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,Hq,Hkv,D,P", [
    ([40000], 8, 1, 128, 64),                       # one unit over many blocks
    ([30011, 3, 0, 9000, 1, 70], 16, 2, 256, 16),   # very unlike
    ([65] * 700, 4, 1, 64, 16),                     # more sequences than blocks and threads
    ([0] * 300 + [5000] + [0] * 300, 4, 1, 128, 32),
    ([1] * 2000, 2, 2, 64, 1)])
def test_splits(dev, kind, lengths, Hq, Hkv, D, P):
    g = rng(dev, len(lengths))
    table, pages = make_table(lengths, P, dev, g)
    cache, k, v = make_cache(pages, P, Hkv, D, kind, dev, g)
    q = (2 * torch.randn((len(lengths), Hq, D), generator=g, device=dev)).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("kind", KINDS)
def test_score_ranges(dev, kind):
    """Scores of hundreds (one token takes all), flat ones, a negative scale, q rows from tiny to huge."""
    g = rng(dev, 5)
    lengths = [300, 1000, 64, 5]
    table, pages = make_table(lengths, 16, dev, g)
    cache, k, v = make_cache(pages, 16, 2, 128, kind, dev, g)
    n = torch.tensor(lengths, dtype=torch.int32, device=dev)
    base = torch.randn((4, 8, 128), generator=g, device=dev)
    for f, scale in ((60.0, None), (0.0, None), (1e-3, None), (1.0, -0.3), (2.0 ** 40, 2.0 ** -43), (2.0 ** -60, 2.0 ** 57)):
        check((base * f).to(torch.bfloat16), cache, k, v, table, n, scale=scale)
    mixed = base * torch.exp2(torch.randint(-20, 3, (4, 8, 1), generator=g, device=dev).float())
    check(mixed.to(torch.bfloat16), cache, k, v, table, n)


@pytest.mark.parametrize("kind", KINDS)
def test_masked_places_may_hold_anything(dev, kind):
    """NaN and infinities behind the lengths, in front of the window and in unused pages change nothing."""
    g = rng(dev, 6)
    lengths = [37, 128, 0, 250]
    table, pages = make_table(lengths, 32, dev, g)
    cache, k, v = make_cache(pages, 32, 2, 128, kind, dev, g)
    q = torch.randn((4, 4, 128), generator=g, device=dev).to(torch.bfloat16)
    n = torch.tensor(lengths, dtype=torch.int32, device=dev)
    for window in (0, 41):
        before = check(q, cache, k, v, table, n, window=window)
        seen = torch.zeros((pages, 32), dtype=torch.bool, device=dev)
        for b, m in enumerate(lengths):
            at = torch.arange(max(0, m - window) if window else 0, m, device=dev)
            seen[table[b].long()[at // 32], at % 32] = True
        for t in (k, v):
            bits = t.view(torch.int16) if kind == "bf16" else t.view(torch.uint8)
            junk = torch.tensor([0x7fc0, 0x7f80, -128] if kind == "bf16" else [0x7f, 0xff, 0x7f], device=dev)
            fill = junk.to(bits.dtype)[torch.randint(0, 3, bits.shape, generator=g, device=dev)]
            bits.copy_(torch.where(seen[:, :, None, None], bits, fill))
        from memory_bound_moe_gb300 import moe_paged_attention
        assert torch.equal(moe_paged_attention(q, cache, table, n, window=window), before)


def test_values_that_are_not_finite(dev):
    g = rng(dev, 7)
    table, pages = make_table([50, 50, 50, 50], 16, dev, g)
    cache, k, v = make_cache(pages, 16, 1, 64, "bf16", dev, g)
    q = torch.randn((4, 2, 64), generator=g, device=dev).to(torch.bfloat16)
    place = lambda b, t: (int(table[b, t // 16]), t % 16, 0)   # noqa: E731
    v[place(0, 3)][5] = math.inf
    v[place(0, 4)][6] = math.nan
    k[place(1, 7)][:] = math.nan
    from memory_bound_moe_gb300 import moe_paged_attention
    out = moe_paged_attention(q, cache, table, torch.full((4,), 50, dtype=torch.int32, device=dev)).float()
    assert (out[0, :, 5] == math.inf).all() and out[0, :, 6].isnan().all()
    assert out[0, :, :5].isfinite().all() and out[0, :, 7:].isfinite().all()
    assert out[1].isnan().all() and out[2:].isfinite().all()


@pytest.mark.parametrize("P", [4, 64])
def test_pages_outside_the_cache_are_left_out(dev, P):
    g = rng(dev, 8)
    lengths = [300, 64, 10, 5]
    table, pages = make_table(lengths, P, dev, g)
    cache, k, v = make_cache(pages, P, 2, 128, "bf16", dev, g)
    q = torch.randn((4, 8, 128), generator=g, device=dev).to(torch.bfloat16)
    table[0, 1], table[0, 3] = -1, pages
    table[1, 0], table[3, :] = -2 ** 31, 2 ** 31 - 1
    out = check(q, cache, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=dev))
    assert (out[3] == 0).all()


def test_lengths_outside_the_table(dev):
    g = rng(dev, 9)
    table, pages = make_table([64, 64, 64], 16, dev, g)
    cache, k, v = make_cache(pages, 16, 1, 64, "bf16", dev, g)
    q = torch.randn((3, 4, 64), generator=g, device=dev).to(torch.bfloat16)
    check(q, cache, k, v, table, torch.tensor([-5, 2 ** 31 - 1, 64], dtype=torch.int32, device=dev))


def test_q_sliced_from_a_projection(dev):
    g = rng(dev, 10)
    lengths = [100, 33, 7]
    table, pages = make_table(lengths, 16, dev, g)
    cache, k, v = make_cache(pages, 16, 2, 128, "bf16", dev, g)
    qkv = torch.randn((3, (8 + 4) * 128), generator=g, device=dev).to(torch.bfloat16)
    q = qkv[:, :8 * 128].unflatten(1, (8, 128))
    n = torch.tensor(lengths, dtype=torch.int32, device=dev)
    a = check(q, cache, k, v, table, n)
    assert torch.equal(a, check(q.contiguous(), cache, k, v, table, n))


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_beyond_32_bits(dev, kind):
    """Three pages, 2^31 and more bytes apart."""
    from memory_bound_moe_gb300 import KVCache
    g = rng(dev, 11)
    P, H, D = 16, 2, 64
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    far = 2 ** 31 + 4096 + 64     # elements
    sides = []
    for _ in range(2):
        flat = torch.empty(2 * far + P * H * D, dtype=dt, device=dev)
        t = flat.as_strided((3, P, H, D), (far, H * D, D, 1))
        t.copy_(torch.randn(t.shape, generator=g, device=dev).to(dt))
        sides.append(t)
    k, v = sides
    q = torch.randn((2, 4, D), generator=g, device=dev).to(torch.bfloat16)
    table = torch.tensor([[2, 0, 1], [1, 2, 0]], dtype=torch.int32, device=dev)
    check(q, KVCache(k, v), k, v, table, torch.tensor([48, 41], dtype=torch.int32, device=dev))


def test_nothing_to_do_and_buffers(dev):
    from memory_bound_moe_gb300 import moe_paged_attention, moe_paged_attention_workspace_size
    g = rng(dev, 12)
    cache, k, v = make_cache(4, 16, 2, 64, "bf16", dev, g)
    empty = moe_paged_attention(torch.empty((0, 4, 64), dtype=torch.bfloat16, device=dev), cache,
                                torch.empty((0, 3), dtype=torch.int32, device=dev), torch.empty(0, dtype=torch.int32, device=dev))
    assert empty.shape == (0, 4, 64)
    # a workspace full of NaN, and not a byte written behind it
    n = moe_paged_attention_workspace_size(2, 4, 2, 64)
    ws = torch.full((n + 64,), 0xff, dtype=torch.uint8, device=dev)
    q = torch.randn((2, 4, 64), generator=g, device=dev).to(torch.bfloat16)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=dev)
    check(q, cache, k, v, table, torch.tensor([32, 20], dtype=torch.int32, device=dev), workspace=ws[:n])
    assert (ws[n:] == 0xff).all()


def test_streams_graphs_and_a_shared_workspace(dev):
    """A captured call replayed over changing lengths, between eager calls that use the same workspace."""
    from memory_bound_moe_gb300 import moe_paged_attention, moe_paged_attention_workspace_size
    g = rng(dev, 13)
    table, pages = make_table([4000, 4000], 16, dev, g)
    cache, k, v = make_cache(pages, 16, 2, 128, "bf16", dev, g)
    q = torch.randn((2, 8, 128), generator=g, device=dev).to(torch.bfloat16)
    lengths = torch.tensor([4000, 4000], dtype=torch.int32, device=dev)
    ws = torch.empty(moe_paged_attention_workspace_size(2, 8, 2, 128), dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    call = lambda **kw: moe_paged_attention(q, cache, table, lengths, workspace=ws, **kw)   # noqa: E731
    eager = call().clone()
    torch.cuda.synchronize()
    other = call(stream=side)
    side.synchronize()
    assert torch.equal(other, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out=out)
    for n in ([4000, 4000], [1, 0], [17, 3999], [0, 0], [2500, 64]):
        lengths.copy_(torch.tensor(n, dtype=torch.int32))
        want = check(q, cache, k, v, table, lengths, workspace=ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
