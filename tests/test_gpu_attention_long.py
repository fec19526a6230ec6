"""Paged attention of long sequences, in bounds that a few tokens left out or
taken twice would pass (test_attention_bounds_cpu.py)."""
from __future__ import annotations

import math

import pytest
import torch

import attention_bounds as bounds
from test_gpu_attention_paths import widened
from test_gpu_paged_attention import KINDS, dev, make_cache, make_table, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,Hq,Hkv,D,P,wide", [
    ([40000], 8, 1, 128, 64, 0),
    ([1000003, 5], 3, 1, 64, 1024, 0),
    ([1000003, 70000], 3, 1, 64, 16, 0),
    ([131072, 1, 70001], 8, 4, 64, 64, 0),                     # four heads side by side
    ([30011, 3, 0, 9000, 1, 70], 16, 2, 256, 16, 0),
    ([20000, 3, 777], 40, 1, 64, 32, 0),                       # three groups of 16 heads
    ([20000, 3, 777], 64, 1, 128, 32, 0),                      # four, side by side
    ([(37 * i) % 5000 for i in range(64)], 16, 8, 128, 1, 0),  # many units a run
    ([700] * 9, 8, 2, 128, 16, 0),                             # clusters
    ([700] * 9, 8, 2, 128, 16, 200000),                        # the same in a wide table
    ([3900, 64, 2047], 16, 1, 256, 8, 0)])
def test_every_token_counts_once(dev, kind, lengths, Hq, Hkv, D, P, wide):  # noqa: F811
    from memory_bound_moe_gb300 import KVCache, moe_paged_attention
    g = rng(dev, len(lengths))
    table, pages = make_table(lengths, P, dev, g)
    t = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    k, v = (torch.empty((pages, P, Hkv, D), dtype=t, device=dev) for _ in "kv")
    k.copy_(torch.randn((P, Hkv, D), generator=g, device=dev).to(t).expand(pages, P, Hkv, D))
    cache, given = KVCache(k, v), widened(table, P, wide) if wide else table
    q = torch.zeros((len(lengths), Hq, D), dtype=torch.bfloat16, device=dev)
    n32 = torch.tensor(lengths, dtype=torch.int32, device=dev)
    chain = bounds.chain(lengths, Hkv, Hq // Hkv, sms())
    R = max(bounds.passes(n, D) for n in lengths)
    for r in range(R):
        v.view(torch.int16 if kind == "bf16" else torch.uint8).zero_()
        want = torch.zeros((len(lengths), Hkv, D), dtype=torch.float64, device=dev)
        for b, n in enumerate(lengths):
            at = torch.arange(n, device=dev)
            page = table[b].long()[at // P]
            for h in range(Hkv):
                cols = bounds.column(n, D, R, r, h, dev)
                here = cols >= 0
                one = torch.ones((), dtype=t, device=dev)
                v.view(torch.int16 if kind == "bf16" else torch.uint8)[page[here], at[here] % P, h, cols[here]] = one.view(
                    torch.int16 if kind == "bf16" else torch.uint8)
                want[b, h] = bounds.counted(cols, D) / max(1, n)
        lse = torch.empty((len(lengths), Hq), device=dev)
        out = moe_paged_attention(q, cache, given, n32, lse=lse).double().view(len(lengths), Hkv, -1, D)
        tol = bounds.counted_tol(want, chain, kind == "e4m3")
        off = (out - want[:, :, None]).abs()
        assert (off <= tol[:, :, None]).all(), f"pass {r}: {float((off / tol[:, :, None].clamp_min(1e-300)).max()):.3g} of the bound"
        for b, n in enumerate(lengths):
            if n == 0:
                assert (lse[b] == -math.inf).all()
            else:
                assert (lse[b].double() - math.log(n)).abs().max() <= bounds.counted_lse_tol(n, chain, kind == "e4m3")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,Hq,Hkv,D,P,window", [
    ([40000], 4, 1, 64, 64, 0),
    ([40000], 16, 1, 128, 16, 0),
    ([70000, 5], 4, 1, 64, 32, 0),
    ([30011, 3, 0, 9000, 1, 70], 16, 2, 256, 16, 0),
    ([30011, 3, 0, 9000, 1, 70], 16, 4, 128, 1, 7001),
    ([65] * 700, 4, 1, 64, 16, 0),
    ([0] * 300 + [5000] + [0] * 300, 4, 1, 128, 32, 0),
    ([20000, 3], 64, 1, 64, 16, 0),
    ([(53 * i) % 3000 for i in range(48)], 32, 8, 64, 16, 0)])
def test_random_sequences(dev, kind, lengths, Hq, Hkv, D, P, window):  # noqa: F811
    from memory_bound_moe_gb300 import moe_paged_attention
    g = rng(dev, len(lengths) + D)
    table, pages = make_table(lengths, P, dev, g)
    cache, k, v = make_cache(pages, P, Hkv, D, kind, dev, g)
    q = ((0.1 if kind == "bf16" else 0.1 / 0.84) * torch.randn((len(lengths), Hq, D), generator=g, device=dev)).to(torch.bfloat16)
    chain = bounds.chain([min(n, window or n) for n in lengths], Hkv, Hq // Hkv, sms())
    f32 = lambda x: float(torch.tensor(x, dtype=torch.float32))   # noqa: E731
    want, want_lse, tol, ltol = bounds.attention(q, k, v, table, lengths, f32(D ** -0.5), chain, window, f32(cache.k_scale),
                                                 f32(cache.v_scale))
    lse = torch.empty((len(lengths), Hq), device=dev)
    out = moe_paged_attention(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device=dev), window=window, lse=lse)
    off = (out.double() - want).abs()
    assert (off <= tol).all(), f"out: {float((off / tol.clamp_min(1e-300)).max()):.3g} of the bound"
    there = want_lse.isfinite()
    loff = (lse.double() - want_lse)[there].abs()
    assert (loff <= ltol[there]).all(), f"lse: {float((loff / ltol[there]).max()):.3g} of the bound"
    assert (lse[~there] == -math.inf).all() and (out[~there] == 0).all()
