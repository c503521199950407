"""Layouts that the unquantised products have to accept, on the host under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only; no device code is compiled)."""

import os

import pytest

from test_host_sanitizers import HERE, ROCM_INCLUDE, ROOT, SAN, _build_and_run, _compiler


def test_matmul_layouts_under_asan_and_ubsan(tmp_path):
    gxx = _compiler("g++")
    if not os.path.exists(os.path.join(ROCM_INCLUDE, "hip", "hip_runtime_api.h")):
        pytest.skip("HIP headers not available")
    csrc = os.path.join(ROOT, "quantized_expert_gemv_moe_amd", "csrc")
    exe = str(tmp_path / "matmul_layouts")
    cmd = [gxx, "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
           "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "matmul_abi.cpp"),
           os.path.join(HERE, "host_sanitize", "matmul_layouts.cpp"), "-o", exe]
    assert "matmul layouts ok" in _build_and_run(cmd, exe)
