"""The host checks of the scored router, the integer products and the quantisation of rows under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only; no device code is compiled)."""

import os

import pytest

host = pytest.importorskip("test_host_sanitizers")


def test_integer_and_router_checks_under_asan_and_ubsan(tmp_path):
    gxx = host._compiler("g++")
    if not os.path.exists(os.path.join(host.ROCM_INCLUDE, "hip", "hip_runtime_api.h")):
        pytest.skip("HIP headers not available")
    csrc = os.path.join(host.ROOT, "quantized_expert_gemv_moe_amd", "csrc")
    exe = str(tmp_path / "int_checks")
    sources = [os.path.join(csrc, f) for f in ("matmul_abi.cpp", "matmul_int_abi.cpp", "router_abi.cpp")]
    cmd = [gxx, "-std=c++17", *host.SAN, "-D__HIP_PLATFORM_AMD__", "-I", host.ROCM_INCLUDE, "-I",
           os.path.join(host.ROOT, "include"), "-I", csrc, *sources,
           os.path.join(host.HERE, "host_sanitize", "int_checks.cpp"), "-o", exe]
    assert "integer and router checks ok" in host._build_and_run(cmd, exe)
