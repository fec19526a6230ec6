"""Refusals of the paged cache's entry points without a GPU (fake addresses
that are never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest

from test_abi_cpu import A, INVALID, MISALIGNED, OK, UNSUPPORTED, WORKSPACE, lib, nogpu  # noqa: F401


def cache(k=A[0], v=A[1], pages=4, page=16, heads=2, dim=64, kind=0, strides=None, ks=1.0, vs=1.0):
    from memory_bound_moe_gb300.binding import _CacheStruct
    strides = strides or (page * heads * dim, heads * dim, dim) * 2
    return _CacheStruct(k, v, pages, page, heads, dim, kind, *strides, ks, vs)


BAD_CACHES = [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(pages=0), INVALID), (dict(heads=0), INVALID), (dict(page=0), INVALID),
    (dict(kind=2), INVALID), (dict(page=24), UNSUPPORTED), (dict(page=2048), UNSUPPORTED), (dict(dim=96), UNSUPPORTED),
    (dict(heads=1025), UNSUPPORTED), (dict(pages=2 ** 31), UNSUPPORTED), (dict(ks=0.5), INVALID),
    (dict(kind=1, ks=0.0), INVALID), (dict(kind=1, vs=float("nan")), INVALID), (dict(kind=1, vs=float("inf")), INVALID),
    (dict(kind=1, ks=-1.0), INVALID), (dict(kind=1, ks=1e-40), INVALID), (dict(kind=1, ks=2.0 ** 127), INVALID),
    (dict(k=A[0] + 8), MISALIGNED), (dict(v=A[1] + 2), MISALIGNED), (dict(strides=(2048, 128, 68, 2048, 128, 64)), MISALIGNED),
    (dict(kind=1, strides=(2048, 128, 64, 2048, 136, 64)), MISALIGNED), (dict(strides=(-2048, 128, 64, 2048, 128, 64)), INVALID),
    (dict(strides=(2 ** 60, 128, 64, 2048, 128, 64)), UNSUPPORTED)]


def attention(lib, c=None, q=A[2], qs=256, B=3, heads=4, table=A[3], most=8, lengths=A[4], window=0, scale=0.1, out=A[5], lse=A[6],  # noqa: F811
              ws=A[7], n=1 << 30):
    c = cache() if c is None else c
    return lib.moe_paged_attention(q, qs, B, heads, ctypes.addressof(c), table, most, lengths, window, scale, out, lse, ws, n, None)


def append(lib, c=None, q=A[2], qs=256, k=A[3], ks=128, v=A[4], vs=128, N=5, heads=4, pos=A[5], slots=A[6], cs=A[7], rows=100,  # noqa: F811
           rot=64, qo=A[8], qos=256, ko=A[9], kos=128):
    c = cache() if c is None else c
    return lib.moe_kv_append(q, qs, k, ks, v, vs, N, heads, pos, slots, cs, rows, rot, 0, ctypes.addressof(c), qo, qos, ko, kos, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_cache_rules(lib, nogpu, bad, status):  # noqa: F811
    assert attention(lib, cache(**bad)) == status and append(lib, cache(**bad)) == status


def test_attention_rules(lib, nogpu):  # noqa: F811
    call = lambda **kw: attention(lib, **kw)   # noqa: E731
    assert lib.moe_paged_attention(A[2], 256, 3, 4, None, A[3], 8, A[4], 0, 0.1, A[5], A[6], A[7], 1 << 30, None) == INVALID
    assert call(B=-1) == INVALID and call(heads=0) == INVALID and call(heads=3) == INVALID and call(most=0) == INVALID
    assert call(window=-1) == INVALID and call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(heads=1026) == UNSUPPORTED and call(B=1 << 24) == UNSUPPORTED and call(most=(1 << 26) + 1) == UNSUPPORTED
    assert call(qs=255) == INVALID and call(qs=260) == MISALIGNED and call(qs=1 << 31) == UNSUPPORTED
    for name in ("q", "table", "lengths", "out"):
        assert call(**{name: 0}) == INVALID, name
    for name, a in (("q", A[2]), ("table", A[3]), ("lengths", A[4]), ("out", A[5]), ("lse", A[6]), ("ws", A[7])):
        assert call(**{name: a + 2}) == MISALIGNED, name
    need = ctypes.c_size_t(0)
    assert lib.moe_paged_attention_workspace_size(3, 4, 2, 64, ctypes.byref(need)) == OK and need.value > 0
    assert call(ws=0) == WORKSPACE and call(n=need.value - 1) == WORKSPACE
    for over in (A[0] + 4096, A[1], A[2] + 512, A[3], A[4]):
        assert call(out=over) == INVALID and call(ws=over) == INVALID and call(lse=over) == INVALID, over
    assert call(out=A[7]) == INVALID and call(lse=A[5]) == INVALID
    assert call(B=0, q=0, table=0, lengths=0, out=0, lse=0, ws=0, n=0) == OK


def test_attention_workspace_rules(lib):  # noqa: F811
    size = lambda *a: lib.moe_paged_attention_workspace_size(*a, ctypes.byref(ctypes.c_size_t(0)))   # noqa: E731
    assert size(0, 4, 2, 64) == OK and size(-1, 4, 2, 64) == INVALID and size(1, 3, 2, 64) == INVALID
    assert size(1, 4, 0, 64) == INVALID and size(1, 4, 2, 80) == UNSUPPORTED and size(1, 2048, 2, 64) == UNSUPPORTED
    assert lib.moe_paged_attention_workspace_size(1, 4, 2, 64, None) == INVALID


def test_append_rules(lib, nogpu):  # noqa: F811
    call = lambda **kw: append(lib, **kw)   # noqa: E731
    assert lib.moe_kv_append(A[2], 256, A[3], 128, A[4], 128, 5, 4, A[5], A[6], A[7], 100, 64, 0, None, A[8], 256, 0, 0, None) == INVALID
    assert call(N=-1) == INVALID and call(heads=-1) == INVALID and call(rot=-16) == INVALID and call(rot=80) == INVALID
    assert call(rot=40) == MISALIGNED and call(rows=0) == INVALID and call(rows=-1) == INVALID
    assert call(N=1 << 31) == UNSUPPORTED and call(heads=1025) == UNSUPPORTED
    for name in ("q", "k", "v", "pos", "slots", "cs", "qo"):
        assert call(**{name: 0}) == INVALID, name
    for name in ("qs", "ks", "vs", "qos", "kos"):
        assert call(**{name: 120}) == INVALID, name
        assert call(**{name: 260}) == MISALIGNED, name
    for name, a in (("q", A[2]), ("k", A[3]), ("v", A[4]), ("pos", A[5]), ("slots", A[6]), ("cs", A[7]), ("qo", A[8]), ("ko", A[9])):
        assert call(**{name: a + 2}) == MISALIGNED, name
    assert call(slots=A[6] + 4) == MISALIGNED
    # over the cache, over other inputs, shifted against themselves, over each other
    for name in ("q", "k", "v", "pos", "slots", "cs", "qo", "ko"):
        assert call(**{name: A[0] + 1024}) == INVALID and call(**{name: A[1]}) == INVALID, name
    for over in (A[3], A[4], A[5], A[6], A[7], A[2] + 512):
        assert call(qo=over) == INVALID, over
    for over in (A[2], A[4], A[5], A[6], A[7], A[8], A[3] + 256):
        assert call(ko=over) == INVALID, over
    # slices of one projection: rows of 512, q | k | v; q_out over k's or v's columns
    sliced = dict(q=A[2], k=A[2] + 512, v=A[2] + 768, qs=512, ks=512, vs=512)
    assert call(**sliced, qo=A[2] + 256, qos=512) == INVALID and call(**sliced, qo=A[2] + 512, qos=512) == INVALID
    assert call(**sliced, ko=A[2] + 768, kos=512) == INVALID and call(**sliced, qo=A[2], qos=256) == INVALID
    assert call(N=0, q=0, k=0, v=0, pos=0, slots=0, cs=0, qo=0, ko=0) == OK


def test_page_table_rules(lib, nogpu):  # noqa: F811
    base = dict(c=A[0], a=A[1], B=4, P=16, M=8, N=32, f=A[2], F=64, fc=A[3], t=A[4], l=A[5], s=A[6], p=A[7], sl=A[8], fo=A[9], r=0)

    def call(**kw):
        x = {**base, **kw}
        return lib.moe_page_table(x["c"], x["a"], x["B"], x["P"], x["M"], x["N"], x["f"], x["F"], x["fc"], x["t"], x["l"], x["s"],
                                  x["p"], x["sl"], x["fo"], x["r"], None)
    assert call(B=-1) == INVALID and call(P=0) == INVALID and call(M=0) == INVALID and call(N=-1) == INVALID and call(F=-1) == INVALID
    assert call(P=12) == UNSUPPORTED and call(P=2048) == UNSUPPORTED and call(M=(1 << 26) + 1) == UNSUPPORTED
    assert call(B=16385) == UNSUPPORTED and call(N=1 << 31) == UNSUPPORTED and call(F=1 << 31) == UNSUPPORTED
    for name in ("c", "a", "f", "fc", "t", "l", "s", "p", "sl", "fo"):
        assert call(**{name: 0}) == INVALID, name
        assert call(**{name: base[name] + 2}) == MISALIGNED, name
    assert call(sl=A[8] + 4) == MISALIGNED and call(r=A[9] + 66) == MISALIGNED
    for out in ("t", "l", "s", "p", "sl", "fo", "r"):
        for over in (A[1], A[2] + 128):
            assert call(**{out: over}) == INVALID, (out, over)
    for out in ("t", "s", "p", "sl", "r"):
        assert call(**{out: A[0]}) == INVALID and call(**{out: A[3]}) == INVALID, out
    assert call(l=A[0] + 4) == INVALID and call(l=A[3]) == INVALID and call(fo=A[0]) == INVALID and call(s=A[5] + 8) == INVALID


def test_page_release_rules(lib, nogpu):  # noqa: F811
    base = dict(x=A[0], B=4, P=16, M=8, t=A[1], l=A[2], f=A[3], F=64, fc=A[4])

    def call(**kw):
        y = {**base, **kw}
        return lib.moe_page_release(y["x"], y["B"], y["P"], y["M"], y["t"], y["l"], y["f"], y["F"], y["fc"], None)
    assert call(B=-1) == INVALID and call(P=3) == UNSUPPORTED and call(M=0) == INVALID and call(F=-1) == INVALID
    assert call(B=16385) == UNSUPPORTED and call(F=1 << 31) == UNSUPPORTED
    for name in ("x", "t", "l", "f", "fc"):
        assert call(**{name: 0}) == INVALID, name
        assert call(**{name: base[name] + 2}) == MISALIGNED, name
    for out in ("l", "f", "fc"):
        assert call(**{out: A[0]}) == INVALID and call(**{out: A[1]}) == INVALID, out
    assert call(f=A[2]) == INVALID and call(fc=A[3] + 16) == INVALID
    assert lib.moe_page_release(0, 0, 16, 8, 0, 0, 0, 0, 0, None) == OK


def test_binding_refuses():
    import torch
    from memory_bound_moe_gb300 import KVCache, moe_page_table
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)   # noqa: E731
    with pytest.raises(ValueError):
        KVCache(z(2, 16, 1, 64), z(2, 16, 1, 64))          # CPU tensors
    with pytest.raises(TypeError):
        KVCache(z(2, 16, 1, 64, dt=torch.float16), z(2, 16, 1, 64, dt=torch.float16))
    with pytest.raises(ValueError):
        KVCache(z(2, 16, 64), z(2, 16, 64))
    n = z(2, dt=torch.int32)
    with pytest.raises(ValueError):
        moe_page_table(n, n, z(2, 3, dt=torch.int32), n, n[:1], 16, 4)
