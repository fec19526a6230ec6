"""Child process of tests/test_zz_few_reset.py: calls of the few-token
operators, and the same calls again after cudaDeviceReset, in a process of its
own. Device memory comes from the CUDA runtime (through ctypes), which the
reset frees; it also unloads the library's device code and with it what was
set for its kernels.

Usage: python few_reset_child.py OUT.npz T
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

_vp, _sz, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
H2D, D2H = 1, 2
NVFP4, MXFP4 = 0, 1


def _loaded_cudart():
    with open("/proc/self/maps") as fh:
        for line in fh:
            path = line.split()[-1]
            if "libcudart.so" in os.path.basename(path):
                return ctypes.CDLL(path)
    raise RuntimeError("libcudart is not loaded")


def main():
    out_path, T = sys.argv[1], int(sys.argv[2])
    from memory_bound_moe_gb300.binding import load_library
    lib = load_library()
    rt = _loaded_cudart()
    rt.cudaMalloc.argtypes = [ctypes.POINTER(_vp), _sz]
    rt.cudaMemcpy.argtypes = [_vp, _vp, _sz, _int]
    rt.cudaGetErrorString.restype = ctypes.c_char_p
    rt.cudaGetErrorString.argtypes = [_int]

    def check(err, what):
        if err != 0:
            raise RuntimeError(f"{what}: {rt.cudaGetErrorString(err).decode()}")

    E, k, H, I, N = 4, 2, 128, 64, 40
    rng = np.random.default_rng(5)
    bf = lambda *s: (rng.standard_normal(s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    u8 = lambda *s: rng.integers(0, 256, s, dtype=np.uint8)
    sc = lambda *s: rng.integers(118, 125, s, dtype=np.uint8)   # E4M3 224 to 384, E8M0 2^-9 to 2^-3
    host = {"x": bf(T, H), "logits": rng.standard_normal((T, E)).astype(np.float32), "w": bf(H), "w13": bf(E, 2 * I, H),
            "w2": bf(E, H, I), "c13": u8(E, 2 * I, H // 2), "s13": sc(E, 2 * I, H // 16), "c2": u8(E, H, I // 2),
            "s2": sc(E, H, I // 16), "g": np.full(E, 500.0, np.float32), "codes": u8(N, H // 2), "scales": sc(N, H // 16)}
    need = _sz(0)
    if lib.moe_layer_workspace_size(T, E, k, H, I, ctypes.byref(need)) != 0:
        raise RuntimeError("moe_layer_workspace_size")
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
        ws, y = alloc(need.value), alloc(2 * T * N)
        norm, out, outn, outm = (alloc(2 * T * H) for _ in range(4))
        calls = {
            "norm": (norm, T * H, lib.moe_add_rmsnorm(d["x"], 0, T, H, d["w"], 0.0, 1e-6, norm, 0, None)),
            "gemv": (y, T * N, lib.moe_gemv_fp4(d["x"], T, H, d["codes"], d["scales"], N, NVFP4, 500.0, y, 0, None)),
            "layer": (out, T * H, lib.moe_layer(d["logits"], T, E, k, 1, d["x"], H, I, d["w13"], d["w2"], out, 0, 0, ws,
                                                need.value, None)),
            "nvfp4": (outn, T * H, lib.moe_layer_fp4(d["logits"], T, E, k, 1, d["x"], H, I, NVFP4, d["c13"], d["s13"], d["g"],
                                                     d["c2"], d["s2"], d["g"], outn, 0, 0, ws, need.value, None)),
            "mxfp4": (outm, T * H, lib.moe_layer_fp4(d["logits"], T, E, k, 1, d["x"], H, I, MXFP4, d["c13"], d["s13"], 0,
                                                     d["c2"], d["s2"], 0, outm, 0, 0, ws, need.value, None)),
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
    np.savez(out_path, **saved)


if __name__ == "__main__":
    main()
