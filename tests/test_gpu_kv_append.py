"""Rotary embedding with the cache's writes, against float64."""
from __future__ import annotations

import pytest
import torch

import cache_reference as ref
from test_gpu_paged_attention import KINDS, dev, make_cache, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def angles(rows, rot, dev):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / max(1, rot))
    a = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def inputs(N, Hq, Hkv, D, pages, P, dev, g, sliced=False):
    if sliced:
        row = torch.randn((N, (Hq + 2 * Hkv) * D + 64), generator=g, device=dev).to(torch.bfloat16)
        q, k, v, _ = row.split([Hq * D, Hkv * D, Hkv * D, 64], 1)
        q, k, v = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
    else:
        q, k, v = (torch.randn((N, h, D), generator=g, device=dev).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    slots = torch.randperm(pages * P, generator=g, device=dev)[:N].contiguous()
    positions = torch.randint(0, 5000, (N,), generator=g, device=dev).int()
    return q, k, v, slots, positions


def check(cache, kc, vc, q, k, v, positions, slots, cos_sin, interleaved=False, keep=None, **kw):
    """One call against the definitions; `keep`: the tokens that are not left out. Returns (q_out, k_out)."""
    from memory_bound_moe_gb300 import moe_kv_append
    N = k.shape[0]
    keep = torch.ones(N, dtype=torch.bool, device=k.device) if keep is None else keep
    e4m3 = kc.dtype == torch.float8_e4m3fn
    P = kc.shape[1]
    q0, k0, v0 = (None if t is None else t.clone() for t in (q, k, v))
    kc0, vc0 = kc.double(), vc.double()
    q_out, k_out = kw.get("q_out"), kw.get("k_out")
    before = {n: t.clone() for n, t in (("q", q_out), ("k", k_out)) if t is not None}
    got = moe_kv_append(q, k, v, positions, slots, cos_sin, cache, interleaved=interleaved, **kw)
    pos = positions[keep] if cos_sin is not None else torch.zeros(int(keep.sum()), device=k.device)
    cs = cos_sin if cos_sin is not None else torch.zeros((1, 0), device=k.device)
    for name, out, src in (("q", got, q0), ("k", k_out, k0)):
        if out is None or src is None:
            continue
        y, err = ref.rotate(src[keep], cs, pos, interleaved)
        want, tol = ref.cached_values(y, err, 1.0, False)
        assert ((out[keep].double() - want).abs() <= tol).all(), name
        if name in before:
            assert torch.equal(out[~keep], before[name][~keep])
    at = (slots[keep] // P, slots[keep] % P)
    for name, c, c0, x, scale in (("k", kc, kc0, k0, cache.k_scale), ("v", vc, vc0, v0, cache.v_scale)):
        y, err = ref.rotate(x[keep], cs if name == "k" else cs[:, :0], pos, interleaved)
        want, tol = ref.cached_values(y, err, scale, e4m3)
        full, bound = c0.clone(), torch.zeros_like(c0)
        full[at], bound[at] = want, tol
        off = (c.double() - full).abs()
        assert (off <= bound).all(), f"{name} cache: {float((off - bound).max())}"   # 0 off where no token went
    return got, k_out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 0), (128, 128), (128, 48), (256, 256), (256, 64), (256, 240)])
@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (7, 16, 2), (300, 5, 5)])
def test_forms(dev, kind, interleaved, D, rot, N, Hq, Hkv):  # noqa: F811
    g = rng(dev, D + rot + N)
    pages, P = 40, 16
    cache, kc, vc = make_cache(pages, P, Hkv, D, kind, dev, g)
    q, k, v, slots, positions = inputs(N, Hq, Hkv, D, pages, P, dev, g)
    cs = angles(5000, rot, dev) if rot else None
    check(cache, kc, vc, q, k, v, positions if rot else None, slots, cs, interleaved)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["token", "head", "joint"])
@pytest.mark.parametrize("P", [1, 8, 64])
def test_layouts_slices_and_in_place(dev, kind, layout, P):  # noqa: F811
    g = rng(dev, P)
    N, Hq, Hkv, D, pages = 33, 6, 3, 128, 64
    cache, kc, vc = make_cache(pages, P, Hkv, D, kind, dev, g, layout)
    cs = angles(5000, D, dev)
    q, k, v, slots, positions = inputs(N, Hq, Hkv, D, pages, P, dev, g, sliced=True)
    apart, k_apart = check(cache, kc, vc, q, k, v, positions, slots, cs, k_out=torch.empty((N, Hkv, D), dtype=torch.bfloat16, device=dev))
    v0 = v.clone()
    first = (kc.clone(), vc.clone())
    got, k_out = check(cache, kc, vc, q, k, v, positions, slots, cs, q_out=q, k_out=k)
    assert got is q and torch.equal(q, apart) and torch.equal(k, k_apart) and torch.equal(v, v0)
    assert torch.equal(kc.view(torch.uint8), first[0].view(torch.uint8)) and torch.equal(vc.view(torch.uint8), first[1].view(torch.uint8))


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_left_out(dev, kind):  # noqa: F811
    """Slots and positions outside their ranges: rows and cache stay as they were."""
    g = rng(dev, 3)
    N, Hq, Hkv, D, pages, P = 40, 4, 2, 64, 8, 8
    cache, kc, vc = make_cache(pages, P, Hkv, D, kind, dev, g)
    q, k, v, slots, positions = inputs(N, Hq, Hkv, D, pages, P, dev, g)
    keep = torch.ones(N, dtype=torch.bool, device=dev)
    for i, s in ((0, -1), (5, pages * P), (6, 2 ** 62), (7, -2 ** 63), (39, -1)):
        slots[i], keep[i] = s, False
    for i, p in ((9, -1), (10, 5000), (11, 2 ** 31 - 1)):
        positions[i], keep[i] = p, False
    q_out = torch.randn((N, Hq, D), generator=g, device=dev).to(torch.bfloat16)
    k_out = torch.randn((N, Hkv, D), generator=g, device=dev).to(torch.bfloat16)
    check(cache, kc, vc, q, k, v, positions, slots, angles(5000, D, dev), keep=keep, q_out=q_out, k_out=k_out)


def test_without_q_and_without_tokens(dev):  # noqa: F811
    from memory_bound_moe_gb300 import moe_kv_append
    g = rng(dev, 4)
    cache, kc, vc = make_cache(8, 16, 2, 64, "bf16", dev, g)
    q, k, v, slots, positions = inputs(20, 4, 2, 64, 8, 16, dev, g)
    check(cache, kc, vc, None, k, v, positions, slots, angles(5000, 64, dev))
    none = moe_kv_append(q[:0], k[:0], v[:0], positions[:0], slots[:0], angles(5000, 64, dev), cache)
    assert none.shape == (0, 4, 64)


def test_e4m3_saturates_and_keeps_nan(dev):  # noqa: F811
    from memory_bound_moe_gb300 import moe_kv_append
    g = rng(dev, 5)
    cache, kc, vc = make_cache(2, 16, 1, 64, "e4m3", dev, g)
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=dev)
    k[0, 0, :6] = torch.tensor([1e30, -1e30, float("inf"), float("-inf"), float("nan"), 448 * 0.021 * 1.01], device=dev)
    moe_kv_append(None, k, k, None, torch.tensor([17], device=dev), None, cache)
    for c in (kc, vc):
        x = c[1, 1, 0].float()
        assert x[:4].tolist() == [448, -448, 448, -448] and x[4].isnan() and (x[6:] == 0).all()
    assert float(kc[1, 1, 0, 5]) == 448


def test_bfloat16_values_are_copied_bit_for_bit(dev):  # noqa: F811
    g = rng(dev, 6)
    from memory_bound_moe_gb300 import moe_kv_append
    cache, kc, vc = make_cache(4, 16, 1, 64, "bf16", dev, g)
    bits = torch.randint(-2 ** 15, 2 ** 15, (64, 1, 64), generator=g, device=dev).to(torch.int16)
    x = bits.view(torch.bfloat16)
    moe_kv_append(x, x.clone(), x.clone(), None, torch.arange(64, device=dev), None, cache)
    assert torch.equal(kc.view(torch.int16).view(64, 1, 64), bits) and torch.equal(vc.view(torch.int16).view(64, 1, 64), bits)


def test_offsets_beyond_32_bits(dev):  # noqa: F811
    from memory_bound_moe_gb300 import KVCache
    g = rng(dev, 7)
    P, H, D, far = 16, 2, 64, 2 ** 31 + 4096
    k_c, v_c = (torch.zeros(far + P * H * D, dtype=torch.bfloat16, device=dev).as_strided((2, P, H, D), (far, H * D, D, 1)) for _ in "kv")
    q, k, v, slots, positions = inputs(20, 4, H, D, 2, P, dev, g)
    check(KVCache(k_c, v_c), k_c, v_c, q, k, v, positions, slots, angles(5000, D, dev))


@pytest.mark.parametrize("N", [1, 16, 4099])
def test_large_and_captured(dev, N):  # noqa: F811
    from memory_bound_moe_gb300 import moe_kv_append
    g = rng(dev, N)
    pages, P, Hq, Hkv, D = 300, 16, 64, 8, 128
    cache, kc, vc = make_cache(pages, P, Hkv, D, "bf16", dev, g)
    q, k, v, slots, positions = inputs(N, Hq, Hkv, D, pages, P, dev, g, sliced=True)
    cs = angles(5000, D, dev)
    want, _ = check(cache, kc, vc, q, k, v, positions, slots, cs)
    k1, v1 = kc.clone(), vc.clone()
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe_kv_append(q, k, v, positions, slots, cs, cache, q_out=out)
    for t in (kc, vc):
        t.view(-1, Hkv, D)[slots] = 0
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, k1) and torch.equal(vc, v1)
