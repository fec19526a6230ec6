"""Child process of tests/test_zz_cache_reset.py: calls of the paged cache's
operators, and the same calls again after cudaDeviceReset, in a process of its
own. Device memory comes from the CUDA runtime (through ctypes), which the
reset frees; it also unloads the library's device code and with it what was
set for its kernels.

Usage: python cache_reset_child.py OUT.npz
Writes the outputs of both rounds (suffixes 0 and 1).
"""
from __future__ import annotations

import ctypes
import os
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
sys.path.insert(0, ROOT)
sys.path.insert(0, HERE)

from few_reset_child import D2H, H2D, _loaded_cudart   # noqa: E402

_vp, _sz, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int


def main():
    from memory_bound_moe_gb300.binding import _CacheStruct, load_library
    lib = load_library()
    rt = _loaded_cudart()
    rt.cudaMalloc.argtypes = [ctypes.POINTER(_vp), _sz]
    rt.cudaMemcpy.argtypes = [_vp, _vp, _sz, _int]
    rt.cudaGetErrorString.restype = ctypes.c_char_p
    rt.cudaGetErrorString.argtypes = [_int]

    def check(err, what):
        if err != 0:
            raise RuntimeError(f"{what}: {rt.cudaGetErrorString(err).decode()}")

    # a narrow table (clusters) and a wide one (runs and their join); 5000 requests need more than 48 KB
    B, Hq, Hkv, D, P, pages, wide, many = 3, 16, 2, 128, 16, 64, 20000, 5000
    rng = np.random.default_rng(5)
    bf = lambda *s: (rng.standard_normal(s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)   # noqa: E731
    ids = rng.permutation(pages).astype(np.int32)
    lengths = np.array([300, 17, 400], np.int32)
    table = np.zeros((B, wide), np.int32)
    for b in range(B):
        table[b, :26] = ids[b * 19:b * 19 + 26]
    angle = rng.uniform(0, 6, (500, D // 2))
    host = {"q": bf(B, Hq, D), "k": bf(B, Hkv, D), "v": bf(B, Hkv, D), "kc": bf(pages, P, Hkv, D), "vc": bf(pages, P, Hkv, D),
            "table": table, "narrow": np.ascontiguousarray(table[:, :26]), "lengths": lengths,
            "slots": np.array([5, 900, 77], np.int64), "positions": np.array([3, 499, 0], np.int32),
            "cs": np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32),
            "cached": rng.integers(0, 30, many).astype(np.int32), "added": np.ones(many, np.int32),
            "many": np.zeros((many, 2), np.int32), "free": np.arange(many, dtype=np.int32), "count": np.array([many], np.int32)}
    need = _sz(0)
    if lib.moe_paged_attention_workspace_size(B, Hq, Hkv, D, ctypes.byref(need)) != 0:
        raise RuntimeError("moe_paged_attention_workspace_size")
    saved = {}
    for rnd in range(2):
        check(rt.cudaSetDevice(0), "cudaSetDevice")

        def alloc(n):
            p = _vp()
            check(rt.cudaMalloc(ctypes.byref(p), n), "cudaMalloc")
            return p.value

        d = {}
        for name, a in host.items():
            d[name] = alloc(a.nbytes)
            check(rt.cudaMemcpy(d[name], a.ctypes.data, a.nbytes, H2D), f"copy {name}")
        ws, qo, out, out_wide = alloc(need.value), alloc(2 * B * Hq * D), alloc(2 * B * Hq * D), alloc(2 * B * Hq * D)
        lens, starts, pos, slots, left = alloc(4 * many), alloc(4 * many + 4), alloc(4 * many), alloc(8 * many), alloc(4)
        cache = _CacheStruct(d["kc"], d["vc"], pages, P, Hkv, D, 0, *((P * Hkv * D, Hkv * D, D) * 2), 1.0, 1.0)
        ref = ctypes.addressof(cache)
        att = lambda t, m, o: lib.moe_paged_attention(qo, Hq * D, B, Hq, ref, t, m, d["lengths"], 0, 0.09, o, 0, ws, need.value, None)   # noqa: E731
        calls = {
            "table": (slots, 4 * many, lib.moe_page_table(d["cached"], d["added"], many, P, 2, many, d["free"], many, d["count"],
                                                          d["many"], lens, starts, pos, slots, left, 0, None)),
            "append": (d["kc"], pages * P * Hkv * D, lib.moe_kv_append(d["q"], Hq * D, d["k"], Hkv * D, d["v"], Hkv * D, B, Hq,
                                                                     d["positions"], d["slots"], d["cs"], 500, D, 0, ref, qo, Hq * D,
                                                                     0, 0, None)),
            "attention": (out, B * Hq * D, att(d["narrow"], 26, out)),
            "runs": (out_wide, B * Hq * D, att(d["table"], wide, out_wide)),
        }
        for name, (_, _, st) in calls.items():
            if st != 0:
                raise RuntimeError(f"{name} returned status {st} in round {rnd}")
        check(rt.cudaDeviceSynchronize(), "cudaDeviceSynchronize")
        for name, (p, n, _) in calls.items():
            a = np.empty(n, np.uint16)
            check(rt.cudaMemcpy(a.ctypes.data, p, a.nbytes, D2H), f"copy {name}")
            saved[f"{name}{rnd}"] = a
        check(rt.cudaDeviceReset(), "cudaDeviceReset")      # frees every allocation above
    np.savez(out_path(), **saved)


def out_path():
    return sys.argv[1]


if __name__ == "__main__":
    main()
