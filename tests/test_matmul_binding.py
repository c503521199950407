"""The Python side of the unquantised products, as far as it goes without a GPU."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_and_host_checks_need_no_gpu_build_of_torch():
    """torch builds without a GPU lack these names; the host-only calls work there."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import ctypes
import quantized_expert_gemv_moe_amd as moe
st = moe.LinearStruct(in_features=64, out_features=8, n_groups=1, dtype=1, out_dtype=1, w=4096)
assert moe.lib().moe_linear_check(ctypes.byref(st)) == moe.MOE_OK
print("imported")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
