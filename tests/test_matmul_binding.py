"""The Python side of the unquantised products, as far as it goes without a GPU."""

import os
import subprocess
import sys

import pytest
import torch

import quantized_expert_gemv_moe_amd as moe
from quantized_expert_gemv_moe_amd import _lib

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


class _Described:
    """Stands for a Linear whose weights are nowhere: the workspace sizes read the descriptor only."""

    def __init__(self, **kw):
        self.struct = moe.LinearStruct(in_features=8192, out_features=64, n_groups=1, dtype=moe.MOE_DTYPE_BF16,
                                       out_dtype=moe.MOE_DTYPE_BF16, w=4096, **kw)


@pytest.mark.parametrize("rows", [2 ** 32 + 5, 2 ** 31, -2 ** 32 + 5, -2 ** 31 - 1])
def test_workspace_sizes_refuse_rows_past_32_bits(rows):
    """The ABI would see their low 32 bits: 5 rows for 2 ** 32 + 5."""
    for size in (moe.matmul_workspace_size, moe.grouped_workspace_size):
        assert size(_Described(), 5) > 0
        with pytest.raises(ValueError, match="32 bits"):
            size(_Described(), rows)


@pytest.mark.parametrize("n_experts", [2 ** 32 + 4, -2 ** 32 + 4, -2 ** 31 - 1])
def test_combine_refuses_expert_counts_past_32_bits(n_experts):
    """No tokens, so that nothing would be launched for a count taken for 4."""
    y, idx, w = torch.empty((0, 16)), torch.empty((0, 2), dtype=torch.int32), torch.empty((0, 2))
    with pytest.raises(ValueError, match="32 bits"):
        _lib._combine(y, idx, w, n_experts, None, None, None, 0)


def test_linear_refuses_a_clamp_that_fp32_takes_for_none():
    """1e-50 is zero in the descriptor's fp32, and zero means no clamp."""
    with pytest.raises(ValueError, match="clamp_limit"):
        moe.Linear.from_tensors(torch.zeros((4, 8)), clamp_limit=1e-50)
