"""A decode step as it is used: page table, projections, QK norm, the cache's
writes, attention, output projection, norm with the residual, MoE layer."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import cache_reference as ref
from few_reference import random_fp4
from test_gpu_kv_append import angles
from test_gpu_layer import Layer
from test_gpu_paged_attention import KINDS, dev, make_cache, rng  # noqa: F401

pytestmark = pytest.mark.gpu

B, H, Hq, Hkv, D, P, M, N = 7, 256, 8, 2, 64, 8, 40, 32


class Step:
    """The weights, the state and the buffers of a small decode loop."""

    def __init__(self, kind, dev, seed=1):  # noqa: F811
        from memory_bound_moe_gb300 import moe_layer_workspace_size, moe_paged_attention_workspace_size
        g = rng(dev, seed)
        r = np.random.default_rng(seed)
        w = lambda n, k: tuple(torch.from_numpy(a).to(dev) for a in random_fp4(r, (n, k), "nvfp4"))   # noqa: E731
        self.g, self.dev = g, dev
        self.wq, self.wk, self.wv, self.wo, self.router = w(Hq * D, H), w(Hkv * D, H), w(Hkv * D, H), w(H, Hq * D), w(16, H)
        self.layer = Layer(16, H, 160, "bf16", dev, 61)
        self.norm, self.qw = torch.ones(H, dtype=torch.bfloat16, device=dev), torch.ones(D, dtype=torch.bfloat16, device=dev)
        self.cs = angles(M * P, D, dev)
        self.cache, self.k, self.v = make_cache(200, P, Hkv, D, kind, dev, g)
        i32 = dict(dtype=torch.int32, device=dev)
        self.lengths, self.added, self.finished = (torch.zeros(B, **i32) for _ in range(3))
        self.table = torch.full((B, M), -1, **i32)
        self.free, self.count = torch.randperm(200, generator=g, device=dev).int(), torch.tensor([200], **i32)
        self.ws = torch.empty(moe_paged_attention_workspace_size(B, Hq, Hkv, D), dtype=torch.uint8, device=dev)
        self.ws2 = torch.empty(moe_layer_workspace_size(B, 16, 4, H, 160), dtype=torch.uint8, device=dev)
        self.x = torch.randn((B, H), generator=g, device=dev).to(torch.bfloat16)
        self.residual = torch.zeros_like(self.x)

    def run(self, wait=False, seen=None):
        """One token for every request."""
        import memory_bound_moe_gb300 as moe
        sync = torch.cuda.synchronize if wait else lambda: None
        y, _ = moe.moe_add_rmsnorm(self.x, self.residual, self.norm)
        sync()
        q, k, v = (moe.moe_gemv_fp4(y, *w, "nvfp4", 3e4).view(B, -1, D) for w in (self.wq, self.wk, self.wv))
        sync()
        moe.moe_qk_rmsnorm(q, k, self.qw, self.qw)
        sync()
        self.t = moe.moe_page_table(self.lengths, self.added, self.table, self.free, self.count, P, N)
        sync()
        raw = (q.clone(), k.clone(), v.clone()) if seen is not None else None
        moe.moe_kv_append(q, k, v, self.t.positions[:B], self.t.slots[:B], self.cs, self.cache, q_out=q)
        sync()
        a = moe.moe_paged_attention(q, self.cache, self.table, self.t.lengths, workspace=self.ws)
        sync()
        o = moe.moe_gemv_fp4(a.view(B, Hq * D), *self.wo, "nvfp4", 3e4)
        sync()
        z, _ = moe.moe_add_rmsnorm(o, self.residual, self.norm)
        logits = moe.moe_gemv_fp4(z, *self.router, "nvfp4", 3e4, out_dtype=torch.float32)
        sync()
        self.layer(logits, z, 4, True, out=self.x, workspace=self.ws2)
        sync()
        self.lengths.copy_(self.t.lengths)
        if seen is not None:
            seen.append((raw, q, a))


@pytest.mark.parametrize("kind", KINDS)
def test_steps_against_the_definitions(dev, kind):  # noqa: F811
    s = Step(kind, dev)
    s.added.fill_(1)
    # the last request's row is full: it is refused, and its token left out
    s.table[B - 1] = s.free[-M:]
    s.count -= M
    s.lengths[B - 1] = M * P
    e4m3 = kind == "e4m3"
    for _ in range(3 * P):
        before, kc0, vc0 = s.lengths.clone(), s.k.double(), s.v.double()
        seen = []
        s.run(seen=seen)
        (q0, k0, v0), q, a = seen[0]
        assert s.t.lengths.tolist() == [int(n) + (b < B - 1) for b, n in enumerate(before)] and int(s.t.refused) == 1
        assert s.t.positions[:B - 1].tolist() == before[:B - 1].tolist() and int(s.t.slots[B - 1]) == -1
        pos, slots = s.t.positions[:B - 1], s.t.slots[:B - 1]
        for name, c, c0, x, scale in (("k", s.k, kc0, k0, s.cache.k_scale), ("v", s.v, vc0, v0, s.cache.v_scale)):
            y, err = ref.rotate(x[:B - 1], s.cs if name == "k" else s.cs[:, :0], pos, False)
            want, tol = ref.cached_values(y, err, scale, e4m3)
            full, bound = c0.clone(), torch.zeros_like(c0)
            full[slots // P, slots % P], bound[slots // P, slots % P] = want, tol
            assert ((c.double() - full).abs() <= bound).all(), name
        y, err = ref.rotate(q0[:B - 1], s.cs, pos, False)
        want, tol = ref.cached_values(y, err, 1.0, False)
        assert ((q[:B - 1].double() - want).abs() <= tol).all() and torch.equal(q[B - 1], q0[B - 1])
        want, _, tol, _ = ref.attention(q, s.k, s.v, s.table, s.t.lengths, D ** -0.5, 0, s.cache.k_scale, s.cache.v_scale)
        assert ((a.double() - want).abs() <= tol).all() and s.x.isfinite().all()
    held = [p for row, n in zip(s.table.tolist(), s.lengths.tolist()) for p in row[:-(-n // P)]]
    assert len(set(held)) == len(held) == 200 - int(s.count)


@pytest.mark.parametrize("kind", KINDS)
def test_chained_and_captured_steps(dev, kind):  # noqa: F811
    """The same bits with a wait after every call, without any, and as a replayed graph."""
    def state(s):
        return [t.clone() for t in (s.x, s.residual, s.lengths, s.table, s.count, s.k.view(torch.uint8), s.v.view(torch.uint8))]

    steps = 40
    runs = []
    for mode in ("wait", "chain", "graph"):
        s = Step(kind, dev)
        s.added.fill_(1)
        if mode == "graph":
            keep = state(s)
            graph = torch.cuda.CUDAGraph()
            s.run()     # loads the kernels
            for t, v in zip((s.x, s.residual, s.lengths, s.table, s.count, s.k.view(torch.uint8), s.v.view(torch.uint8)), keep):
                t.copy_(v)
            with torch.cuda.graph(graph):
                s.run()
            for _ in range(steps):
                graph.replay()
        else:
            for _ in range(steps):
                s.run(wait=mode == "wait")
        torch.cuda.synchronize()
        runs.append(state(s))
    assert runs[0][2].tolist() == [steps] * B and runs[0][0].isfinite().all()
    for other in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], other))


def test_prompts_in_chunks_then_tokens(dev):  # noqa: F811
    """Prompts that come in chunks of 32 tokens in all, then a token each; finished requests give their pages back."""
    import memory_bound_moe_gb300 as moe
    s = Step("bf16", dev, 5)
    prompt = [3, 50, 0, 17, 8, 64, 1]
    left = list(prompt)
    while sum(left):
        take, room = [], N
        for n in left:
            take.append(min(n, room))
            room -= take[-1]
        s.added.copy_(torch.tensor(take))
        t = moe.moe_page_table(s.lengths, s.added, s.table, s.free, s.count, P, N)
        q, k, v = (torch.randn((N, h, D), generator=s.g, device=dev).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        moe.moe_kv_append(q, k, v, t.positions, t.slots, s.cs, s.cache)
        s.lengths.copy_(t.lengths)
        left = [a - b for a, b in zip(left, take)]
        assert int(t.refused) == 0 and t.starts.tolist()[-1] == sum(take)
    assert s.lengths.tolist() == prompt
    s.added.fill_(1)
    seen = []
    s.run(seen=seen)
    _, q, a = seen[0]
    want, _, tol, _ = ref.attention(q, s.k, s.v, s.table, s.lengths, D ** -0.5)
    assert ((a.double() - want).abs() <= tol).all()
    s.finished.copy_(torch.tensor([0, 1, 0, 1, 0, 0, 1]))
    used = [-(-(n + 1) // P) for n in prompt]
    count = int(s.count)
    moe.moe_page_release(s.finished, s.table, s.lengths, s.free, s.count, P)
    assert int(s.count) == count + used[1] + used[3] + used[6]
    assert s.lengths.tolist() == [0 if f else n + 1 for n, f in zip(prompt, s.finished.tolist())]


def test_tables_in_place_in_front_of_attention(dev):  # noqa: F811
    """Lengths, table and stack updated in place and read at once by the next call: every step sees its own."""
    import memory_bound_moe_gb300 as moe
    g = rng(dev, 9)
    many, page, steps = 1100, 1, 48
    cache, k, v = make_cache(many * steps, page, 1, 64, "bf16", dev, g)
    q = torch.randn((many, 2, 64), generator=g, device=dev).to(torch.bfloat16)
    ws = torch.empty(moe.moe_paged_attention_workspace_size(many, 2, 1, 64), dtype=torch.uint8, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    added, order = torch.ones(many, **i32), torch.randperm(many * steps, generator=g, device=dev).int()

    def run(wait):
        lengths, table, count = torch.zeros(many, **i32), torch.zeros((many, steps), **i32), torch.tensor([many * steps], **i32)
        out = moe.PageTable(lengths, torch.empty(many + 1, **i32), torch.empty(8192, **i32),
                            torch.empty(8192, dtype=torch.int64, device=dev), count, torch.empty(1, **i32))
        results = torch.empty((steps, many, 2, 64), dtype=torch.bfloat16, device=dev)
        torch.cuda.synchronize()
        for i in range(steps):
            moe.moe_page_table(lengths, added, table, order, count, page, 8192, out=out)
            if wait:
                torch.cuda.synchronize()
            moe.moe_paged_attention(q, cache, table, lengths, workspace=ws, out=results[i])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return results

    want = run(True)
    assert not torch.equal(want[0], want[1]) and want.isfinite().all()
    for _ in range(10):
        assert torch.equal(run(False), want)
