"""Float64 references and error bounds of the products for a few tokens.

Bounds. A float32 sum of n terms loses at most about n * 2^-23 of the sum of
their magnitudes (tensor-core additions may truncate: 2^-23, not 2^-24, each).
A warp adds the products of 16 k at a time, which is 16 additions inside and one
to the running sum; up to 20 splits of k in a block and 8 blocks are added last,
and the widths' tails: n <= K/16 + 16 + 28 + 20. Rounding
to bfloat16 is off by at most half a step, 2^-8 of the value, and by 2^-134 at
the bottom of the range."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = {"nvfp4": 16, "mxfp4": 32}
HALF = 2.0 ** -8


def fsum(K):
    return (K / 16 + 64) * 2.0 ** -23


def e2m1(codes):
    """uint8 [..., n/2] -> float64 [..., n], element 2i in the low nibble."""
    c = np.asarray(codes)
    nib = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    mag = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[nib & 7]
    return np.where(nib & 8, -mag, mag)


def e4m3(b):
    """E4M3 bytes -> float64 (0x7f and 0xff are NaN)."""
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def weights64(codes, scales, fmt, g=1.0):
    """Codes and scales of one matrix (numpy) -> float64 values."""
    s = 2.0 ** (np.asarray(scales).astype(np.float64) - 127) if fmt == "mxfp4" else e4m3(scales) / float(g)
    return e2m1(codes) * np.repeat(s, BLOCK[fmt], axis=-1)


def random_fp4(rng, shape, fmt, spread=3):
    """Random codes and scales of matrices [..., n, k]; scale bytes around the
    middle of the format, `spread` binades to each side."""
    *lead, n, k = shape
    codes = rng.integers(0, 256, (*lead, n, k // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scales = rng.integers(122 - spread, 122 + spread + 1, (*lead, n, k // 32)).astype(np.uint8)
    else:
        scales = rng.integers(0, 0x7f, (*lead, n, k // 16)).astype(np.uint8)   # every finite non-negative value
    return codes, scales


def gemv64(x, w):
    """(reference, sum of magnitudes) of x [T, K] (torch bfloat16) @ w.T."""
    x = x.double().cpu().numpy()
    return x @ w.T, np.abs(x) @ np.abs(w).T


def check_gemv(got, x, w, what=""):
    ref, mag = gemv64(x, w)
    bound = fsum(w.shape[1]) * mag + 2.0 ** -149
    if got.dtype == torch.bfloat16:
        bound = bound * (1 + HALF) + HALF * np.abs(ref) + 2.0 ** -134
    else:
        bound = bound + 2.0 ** -22 * np.abs(ref)   # the tensor scale: a reciprocal and a product
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.isfinite(err).all(), what
    assert (err <= bound).all(), (what, np.argwhere(err > bound)[:4].tolist(), float((err / bound).max()))


def check_layer(out, ids, wts, x, expert_weights, H, I, what=""):
    """out [T, H] against the definition for the routing ids, wts [T, k];
    expert_weights(e) -> (w13 [2I, H], w2 [H, I]) in float64. Elementwise
    against the bound carried through the layer, and in the 2-norm against
    2^-8: the two bfloat16 roundings are independent and each at most
    2^-8 / sqrt(3) of the norm."""
    T, k = ids.shape
    xd = x.double().cpu().numpy()
    ref, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        w13, w2 = expert_weights(int(e))
        for t, j in np.argwhere(ids == e):
            g, u = w13[:I] @ xd[t], w13[I:] @ xd[t]
            dg, du = (fsum(H) * (np.abs(w) @ np.abs(xd[t])) for w in (w13[:I], w13[I:]))
            sg = g / (1 + np.exp(-g))
            a = wts[t, j] * sg * u
            # |silu'| <= 1.1; expf, the quotient and the products: 2^-19
            da = wts[t, j] * (1.1 * dg * np.abs(u) + (np.abs(sg) + 1.1 * dg) * du) + (HALF + 2.0 ** -19) * np.abs(a) + 2.0 ** -134
            ref[t] += w2 @ a
            bound[t] += np.abs(w2) @ (da + k * fsum(I) * (np.abs(a) + da))
    bound += HALF * (np.abs(ref) + bound) + 2.0 ** -134
    got = out.double().cpu().numpy()
    err = np.abs(got - ref)
    assert np.isfinite(err).all(), what
    assert (err <= bound).all(), (what, np.argwhere(err > bound)[:4].tolist(), float((err / bound).max()))
    if T * H >= 1000:
        rel = np.linalg.norm(err) / np.linalg.norm(ref)
        assert rel <= HALF, (what, rel)
