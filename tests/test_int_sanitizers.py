"""The host checks of the scored router, the integer products and the quantisation of rows under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only; no device code is compiled)."""

import os

import pytest

from test_host_sanitizers import HERE, ROCM_INCLUDE, ROOT, SAN, _build_and_run, _compiler


def test_integer_and_router_checks_under_asan_and_ubsan(tmp_path):
    gxx = _compiler("g++")
    if not os.path.exists(os.path.join(ROCM_INCLUDE, "hip", "hip_runtime_api.h")):
        pytest.skip("HIP headers not available")
    csrc = os.path.join(ROOT, "quantized_expert_gemv_moe_amd", "csrc")
    exe = str(tmp_path / "int_checks")
    sources = [os.path.join(csrc, f) for f in ("matmul_abi.cpp", "matmul_int_abi.cpp", "router_abi.cpp")]
    cmd = [gxx, "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE, "-I", os.path.join(ROOT, "include"),
           "-I", csrc, *sources, os.path.join(HERE, "host_sanitize", "int_checks.cpp"), "-o", exe]
    assert "integer and router checks ok" in _build_and_run(cmd, exe)
