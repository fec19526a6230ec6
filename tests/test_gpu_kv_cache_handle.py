"""KVCache: what it refuses when it is made, and that it never goes by values
or memory that its tensors no longer have."""
from __future__ import annotations

import pytest
import torch

from test_gpu_paged_attention import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def zeros(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt, device="cuda:0")


def test_refused_when_made(dev):  # noqa: F811
    from memory_bound_moe_gb300 import KVCache, MoeError
    good = zeros(4, 16, 2, 64)
    e4m3 = zeros(4, 16, 2, 64, dt=torch.float8_e4m3fn)
    odd = zeros(4 * 16 * 2 * 64 + 1)[1:].view(4, 16, 2, 64)                # 2 bytes off a 16-byte boundary
    wide = zeros(4, 16, 2, 68)[..., :64]                                   # heads 68 elements apart
    for k, v in ((zeros(4, 16, 2, 96),) * 2, (zeros(4, 24, 2, 64),) * 2, (zeros(1, 2048, 1, 64),) * 2, (zeros(0, 16, 2, 64),) * 2,
                 (zeros(4, 16, 0, 64),) * 2, (zeros(1, 1, 1025, 64),) * 2, (odd, good), (good, odd), (wide, good)):
        with pytest.raises(MoeError):
            KVCache(k, v)
    for kw in (dict(k_scale=0.5), dict(v_scale=2.0)):
        with pytest.raises(MoeError):
            KVCache(good, good.clone(), **kw)
    for bad in (0.0, -1.0, 1e-40, float("inf"), float("nan"), 2.0 ** 127):
        with pytest.raises(MoeError):
            KVCache(e4m3, e4m3.clone(), bad, 1.0)
        with pytest.raises(MoeError):
            KVCache(e4m3, e4m3.clone(), 1.0, bad)
    with pytest.raises(ValueError):
        KVCache(zeros(4, 16, 2, 128)[..., ::2], good)
    KVCache(good, good.clone())
    KVCache(e4m3, e4m3.clone(), 2.0 ** -126, 2.0 ** 126)
    KVCache(zeros(1, 1, 1, 256), zeros(1, 1, 1, 256))


def test_attributes_cannot_be_set(dev):  # noqa: F811
    from memory_bound_moe_gb300 import KVCache
    k, v = (zeros(4, 16, 2, 64, dt=torch.float8_e4m3fn) for _ in "kv")
    cache = KVCache(k, v, 0.5, 0.25)
    for name, value in (("k_scale", 2.0), ("v_scale", 2.0), ("k", v), ("v", k), ("head_dim", 128), ("heads", 1), ("page_size", 8),
                        ("num_pages", 1), ("device_index", 1)):
        with pytest.raises(AttributeError):
            setattr(cache, name, value)
    assert cache.k is k and cache.v is v and (cache.k_scale, cache.v_scale) == (0.5, 0.25)
    assert (cache.num_pages, cache.page_size, cache.heads, cache.head_dim) == (4, 16, 2, 64)
    cache.layer = 3     # a name of the caller's own

    class Named(KVCache):
        def __init__(self, name, *tensors):
            self.name = name
            super().__init__(*tensors)
            self.used = 0

    named = Named("first", k, v)
    assert (named.name, named.used, cache.layer) == ("first", 0, 3)


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("how", ["data", "set_"])
def test_other_memory_is_refused(dev, side, how):  # noqa: F811
    """(What the tensor held before is kept here, so that no call can reach memory that is no more.)"""
    from memory_bound_moe_gb300 import KVCache, moe_kv_append, moe_paged_attention
    k, v = zeros(4, 16, 2, 64), zeros(4, 16, 2, 64)
    cache = KVCache(k, v)
    q, n = zeros(1, 4, 64), torch.tensor([5], dtype=torch.int32, device=dev)
    table = torch.tensor([[1]], dtype=torch.int32, device=dev)
    new, slots = zeros(1, 2, 64) + 1, torch.tensor([3], device=dev)
    t = k if side == "k" else v
    before = t.detach()
    other = zeros(4, 16, 2, 64)
    if how == "data":
        t.data = other
    else:
        t.set_(other)
    with pytest.raises(ValueError):
        moe_paged_attention(q, cache, table, n)
    with pytest.raises(ValueError):
        moe_kv_append(None, new, new, None, slots, None, cache)
    torch.cuda.synchronize()
    assert (before == 0).all() and (other == 0).all()
    moe_kv_append(None, new, new, None, slots, None, KVCache(k, v))
    assert (k[0, 3] == 1).all() and (v[0, 3] == 1).all() and (t.data_ptr() == other.data_ptr())
