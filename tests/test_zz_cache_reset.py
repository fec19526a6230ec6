"""The paged cache's operators after cudaDeviceReset, in a child process."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_cache_operators_after_device_reset(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_moe_gb300 import build
    build.build()
    out = tmp_path / "reset.npz"
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cache_reset_child.py")
    res = subprocess.run([sys.executable, child, str(out)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-2000:]
    d = np.load(out)
    for name in ("table", "append", "attention", "runs"):
        assert np.array_equal(d[name + "0"], d[name + "1"]) and d[name + "0"].any(), name
    a, b = ((d[n].astype(np.uint32) << 16).view(np.float32) for n in ("attention0", "runs0"))
    assert np.isfinite(a).all() and np.abs(a - b).max() <= 2.0 ** -7 * np.abs(a).max()
