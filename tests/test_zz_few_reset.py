"""The few-token operators in a new CUDA context of the same process."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("T", [3, 12])
def test_calls_after_a_device_reset(tmp_path, T):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_moe_gb300 import build
    build.build()
    out = tmp_path / "out.npz"
    res = subprocess.run([sys.executable, os.path.join(HERE, "few_reset_child.py"), str(out), str(T)],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    got = np.load(out)
    for name in ("norm", "gemv", "layer", "nvfp4", "mxfp4"):
        assert got[f"{name}0"].any() and np.array_equal(got[f"{name}0"], got[f"{name}1"]), name
