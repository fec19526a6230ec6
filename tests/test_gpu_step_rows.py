"""A step in which requests bring no token, one or several: the step's rows are
by token, the attention's by request, and `starts` leads from one to the other."""
from __future__ import annotations

import pytest
import torch

import cache_reference as ref
from test_gpu_kv_append import angles
from test_gpu_paged_attention import KINDS, dev, make_cache, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
def test_rows_by_starts(dev, kind):  # noqa: F811
    import memory_bound_moe_gb300 as moe
    g = rng(dev, 4)
    B, Hq, Hkv, D, P, M, N, pages = 7, 8, 2, 64, 8, 12, 24, 120
    cache, k_pages, v_pages = make_cache(pages, P, Hkv, D, kind, dev, g)
    cs = angles(M * P, D, dev)
    i32 = dict(dtype=torch.int32, device=dev)
    table = torch.full((B, M), -1, **i32)
    stack, count = torch.randperm(pages, generator=g, device=dev).int(), torch.tensor([pages], **i32)
    lengths, finished = torch.zeros(B, **i32), torch.zeros(B, **i32)
    #        prompts                 a token each, some pause     one is released, the first is full
    steps = [[3, 9, 1, 0, 5, 2, 4], [1, 0, 1, 0, 0, 1, 1], [1, 1, 0, 6, 1, 0, 1], [1, 0, 0, 2, 0, 0, 1],
             [1, 3, 0, 2, 0, 1, 30]]   # the last one's tokens end behind the step's rows: refused
    for i, added in enumerate(steps):
        if i == 2:
            finished[4] = 1
            moe.moe_page_release(finished, table, lengths, stack, count, P)
            finished.zero_()
            lengths[0] = M * P      # (whatever its pages hold)
            table[0] = torch.arange(M, device=dev)
        a = torch.tensor(added, **i32)
        before = lengths.clone()
        step = moe.moe_page_table(lengths, a, table, stack, count, P, N)
        q, k, v = (torch.randn((N, h, D), generator=g, device=dev).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        raw = q.clone()
        assert moe.moe_kv_append(q, k, v, step.positions, step.slots, cs, cache, q_out=q) is q
        # a request's last token; one without tokens gets a row that is not its own, and so no tokens to attend over
        last = (step.starts[1:] - 1).clamp(0, N - 1).long()
        out = moe.moe_paged_attention(q[last], cache, table, torch.where(a > 0, step.lengths, 0))
        assert out.isfinite().all()
        start = 0
        for b, n in enumerate(added):
            refused = (i >= 2 and b == 0) or n == 30
            if n == 0:
                assert (out[b] == 0).all()
                continue
            row = start + n - 1
            start += n
            if refused:       # its tokens are not stored, and their rows of q as they were
                assert int(step.lengths[b]) == int(before[b]) and torch.equal(q[row - n + 1:row + 1], raw[row - n + 1:row + 1])
                continue
            assert int(step.lengths[b]) == int(before[b]) + n and int(step.positions[row]) == int(step.lengths[b]) - 1
            y, err = ref.rotate(raw[row:row + 1], cs, step.positions[row:row + 1], False)
            want, tol = ref.cached_values(y, err, 1.0, False)
            assert ((q[row:row + 1].double() - want).abs() <= tol).all()
            want, _, tol, _ = ref.attention(q[row:row + 1], k_pages, v_pages, table[b:b + 1], step.lengths[b:b + 1], D ** -0.5, 0,
                                            cache.k_scale, cache.v_scale)
            assert ((out[b:b + 1].double() - want).abs() <= tol).all()
        assert torch.equal(q[start:], raw[start:]) and int(step.refused) == int(i >= 2) + int(i == 4)
        lengths.copy_(step.lengths)
