"""Refusals of the row-norm entry points without a GPU: fake addresses that
are never dereferenced, because every call fails validation (or has nothing to
do) before a launch."""
from __future__ import annotations

import pytest

from test_abi_cpu import A, INVALID, MISALIGNED, OK, UNSUPPORTED, lib, nogpu  # noqa: F401


def test_add_rmsnorm_rules(lib, nogpu):  # noqa: F811
    def call(x=A[0], r=A[1], T=16, H=256, w=A[2], eps=1e-6, out=A[3], ro=A[4]):
        return lib.moe_add_rmsnorm(x, r, T, H, w, 0.0, eps, out, ro, None)
    assert call(T=-1) == INVALID and call(H=0) == INVALID
    assert call(H=250) == MISALIGNED
    assert call(T=2 ** 31) == UNSUPPORTED
    assert call(eps=-1e-6) == INVALID and call(eps=float("nan")) == INVALID
    assert call(x=0) == INVALID and call(w=0) == INVALID and call(out=0) == INVALID
    assert call(r=0) == INVALID                                   # residual_out without a residual
    for name in ("x", "r", "w", "out", "ro"):
        bad = dict(x=A[0], r=A[1], w=A[2], out=A[3], ro=A[4])[name] + 8
        assert call(**{name: bad}) == MISALIGNED, name
    assert call(out=A[0] + 256) == INVALID                        # out over x
    assert call(out=A[1]) == INVALID                              # out over the residual
    assert call(ro=A[1] + 512) == INVALID                         # shifted against the residual
    assert call(ro=A[3]) == INVALID                               # two outputs
    assert call(x=A[1], ro=A[1]) == INVALID                       # in place over x
    assert call(out=A[2]) == INVALID
    assert lib.moe_add_rmsnorm(0, 0, 0, 256, 0, 0.0, 1e-6, 0, 0, None) == OK


def test_add_rmsnorm_mxfp8_rules(lib, nogpu):  # noqa: F811
    def call(x=A[0], r=A[1], T=16, H=256, w=A[2], eps=1e-6, c=A[3], s=A[4], out=A[5], ro=A[6]):
        return lib.moe_add_rmsnorm_mxfp8(x, r, T, H, w, 0.0, eps, c, s, out, ro, None)
    assert call(H=264) == MISALIGNED                              # H % 32
    assert call(c=0) == INVALID and call(s=0) == INVALID
    assert call(c=A[3] + 8) == MISALIGNED and call(out=A[5] + 8) == MISALIGNED
    assert call(c=A[0]) == INVALID and call(s=A[3] + 4) == INVALID and call(out=A[3]) == INVALID
    assert call(ro=A[1] + 64) == INVALID and call(r=0) == INVALID
    assert call(eps=-1.0) == INVALID
    assert lib.moe_add_rmsnorm_mxfp8(0, 0, 0, 256, 0, 0.0, 1e-6, 0, 0, 0, 0, None) == OK


def test_binding_refuses():
    import torch
    from memory_bound_moe_gb300 import moe_add_rmsnorm
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe_add_rmsnorm(x, None, torch.zeros(16, dtype=torch.bfloat16))   # CPU tensors
    with pytest.raises((TypeError, ValueError)):
        moe_add_rmsnorm(x.float(), None, x[0])
