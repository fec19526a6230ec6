"""Refusals of the products for a few tokens without a GPU (fake addresses
that are never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest

from test_abi_cpu import A, INVALID, MISALIGNED, OK, UNSUPPORTED, WORKSPACE, lib, nogpu  # noqa: F401

NV, MX = 0, 1


def test_gemv_fp4_rules(lib, nogpu):  # noqa: F811
    def call(x=A[0], T=4, K=64, c=A[1], s=A[2], N=100, fmt=MX, g=1.0, y=A[3], f32=0):
        return lib.moe_gemv_fp4(x, T, K, c, s, N, fmt, g, y, f32, None)
    assert call(T=-1) == INVALID and call(K=0) == INVALID and call(N=0) == INVALID
    assert call(T=33) == UNSUPPORTED and call(K=(1 << 20) + 32) == UNSUPPORTED
    assert call(K=48, fmt=NV) == MISALIGNED and call(K=40) == MISALIGNED
    assert call(fmt=2) == INVALID and call(fmt=NV, g=0.0) == INVALID and call(fmt=NV, g=float("nan")) == INVALID
    for name, a in (("x", A[0]), ("c", A[1]), ("s", A[2]), ("y", A[3])):
        assert call(**{name: 0}) == INVALID, name
        assert call(**{name: a + 2}) == MISALIGNED, name
    assert call(y=A[0] + 64) == INVALID and call(y=A[1]) == INVALID and call(y=A[2] + 16) == INVALID
    assert lib.moe_gemv_fp4(0, 0, 64, 0, 0, 100, MX, 1.0, 0, 0, None) == OK


def test_layer_workspace_rules(lib):  # noqa: F811
    def size(T=4, E=8, k=2, H=64, I=96):
        out = ctypes.c_size_t(7)
        return lib.moe_layer_workspace_size(T, E, k, H, I, ctypes.byref(out)), out.value
    st, n = size()
    assert st == OK and n >= 2 * 4 * 2 * 96
    assert size(T=0)[0] == OK
    assert size(T=33)[0] == UNSUPPORTED and size(H=1 << 21)[0] == UNSUPPORTED and size(I=1 << 21)[0] == UNSUPPORTED
    assert size(k=9)[0] == INVALID and size(T=-1)[0] == INVALID and size(E=2000)[0] == UNSUPPORTED
    assert size(H=60)[0] == MISALIGNED and size(I=4)[0] == MISALIGNED and size(H=0)[0] == INVALID
    assert lib.moe_layer_workspace_size(4, 8, 2, 64, 96, None) == INVALID


def test_layer_rules(lib, nogpu):  # noqa: F811
    need = ctypes.c_size_t(0)
    assert lib.moe_layer_workspace_size(4, 8, 2, 64, 96, ctypes.byref(need)) == OK

    def call(l=A[0], T=4, E=8, k=2, x=A[1], H=64, I=96, w13=A[2], w2=A[3], out=A[4], ids=A[5], wt=A[6], ws=A[7],
             n=need.value):
        return lib.moe_layer(l, T, E, k, 1, x, H, I, w13, w2, out, ids, wt, ws, n, None)
    assert call(T=33) == UNSUPPORTED and call(E=1025) == UNSUPPORTED and call(k=0) == INVALID and call(k=9) == INVALID
    assert call(H=60) == MISALIGNED and call(I=100) == MISALIGNED
    for name in ("l", "x", "w13", "w2", "out"):
        assert call(**{name: 0}) == INVALID, name
    for name, a in (("l", A[0]), ("x", A[1]), ("w13", A[2]), ("w2", A[3]), ("out", A[4]), ("ids", A[5]), ("wt", A[6]),
                    ("ws", A[7])):
        assert call(**{name: a + 2}) == MISALIGNED, name
    assert call(ws=0) == WORKSPACE and call(n=need.value - 1) == WORKSPACE
    for over in (A[0], A[1], A[2] + 4096, A[3]):
        assert call(out=over) == INVALID and call(ws=over) == INVALID and call(ids=over) == INVALID
    assert call(out=A[7]) == INVALID and call(wt=A[5]) == INVALID
    assert lib.moe_layer(0, 0, 8, 2, 1, 0, 64, 96, 0, 0, 0, 0, 0, 0, 0, None) == OK


def test_layer_fp4_rules(lib, nogpu):  # noqa: F811
    def call(l=A[0], T=4, E=8, k=2, x=A[1], H=64, I=96, fmt=NV, c13=A[2], s13=A[3], g13=A[4], c2=A[5], s2=A[6],
             g2=A[7], out=A[8], ws=A[9], n=1 << 20):
        return lib.moe_layer_fp4(l, T, E, k, 1, x, H, I, fmt, c13, s13, g13, c2, s2, g2, out, 0, 0, ws, n, None)
    assert call(H=72) == MISALIGNED and call(I=40) == MISALIGNED and call(H=48) == MISALIGNED
    assert call(fmt=3) == INVALID
    for name in ("c13", "s13", "g13", "c2", "s2", "g2", "out", "x", "l"):
        assert call(**{name: 0}) == INVALID, name
    for name, a in (("c13", A[2]), ("s13", A[3]), ("g13", A[4]), ("c2", A[5]), ("s2", A[6]), ("g2", A[7])):
        assert call(**{name: a + 2}) == MISALIGNED, name
    assert call(n=10) == WORKSPACE
    for over in (A[2], A[3], A[4], A[5], A[6], A[7]):
        assert call(out=over) == INVALID, over
    assert lib.moe_layer_fp4(0, 0, 8, 2, 1, 0, 64, 96, MX, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, None) == OK


def test_binding_refuses():
    import torch
    from memory_bound_moe_gb300 import moe_gemv_fp4, moe_layer
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    with pytest.raises(ValueError):
        moe_gemv_fp4(z(2, 64), z(5, 32, dt=torch.uint8), z(5, 4, dt=torch.uint8))       # CPU tensors
    with pytest.raises(ValueError):
        moe_gemv_fp4(z(2, 64), z(5, 32, dt=torch.uint8), z(5, 4, dt=torch.uint8), "fp4")
    with pytest.raises(ValueError):
        moe_layer(z(2, 4, dt=torch.float32), z(2, 64), z(4, 64), z(4, 64, 32), 2, True)
