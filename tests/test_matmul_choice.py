"""Which kernel the library takes for the shapes of the products' GPU tests (CPU only: the rule
is host code).  A rule that is fitted anew may change these; the tests' shapes
then have to follow, so that every kernel stays tested."""

import os
import shutil
import subprocess

import pytest

import matmul_cases as cases

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
DTYPES = {"fp32": 0, "bf16": 1, "fp16": 2}


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("no C++ compiler or HIP headers")
    csrc = os.path.join(ROOT, "quantized_expert_gemv_moe_amd", "csrc")
    exe = str(tmp_path_factory.mktemp("choice") / "choice")
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I",
                    os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "matmul_abi.cpp"),
                    os.path.join(HERE, "matmul_choice.cpp"), "-o", exe], check=True)

    def run(queries):
        """Kernels of (dtype, out dtype, gated, experts or 0, rows, K, N), rows packed."""
        lines = [f"{DTYPES[d]} {DTYPES[o]} {int(g)} {e} {r} {k} {n} {int(k * (4 if d == 'fp32' else 2) % 16 == 0)}"
                 for d, o, g, e, r, k, n in queries]
        out = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, check=True).stdout
        return [(w[0], *map(int, w[1:])) for w in (line.split() for line in out.strip().split("\n"))]

    return run


def test_dense_shapes_reach_their_kernels(choose):
    got = choose([(d, d, g, 0, r, k, n) for d, g, r, k, n, _ in cases.DENSE])
    assert got == [c[-1] for c in cases.DENSE]


def test_grouped_shapes_reach_their_kernels(choose):
    got = choose([(d, o, g, e, t * top, k, n) for d, o, g, e, t, top, k, n, _ in cases.GROUPED])
    assert got == [c[-1] for c in cases.GROUPED]


def test_far_rows_reach_their_kernels(choose):
    dense = [cases.FAR_X, cases.FAR_W]
    assert choose([("bf16", "bf16", False, 0, r, k, n) for r, k, n, _, _ in dense]) == [c[-1] for c in dense]
    far = cases.FAR_GATHERED
    assert choose([("bf16", "bf16", False, e, s, k, n) for e, s, k, n, _, _ in far]) == [c[-1] for c in far]
    for _, slots, _, _, stride, _ in far:
        assert 4.25e9 < slots * stride * 2 < 2 ** 32 - 1 and stride % 8 == 0


def test_long_inputs_go_in_stretches(choose):
    for rows, k, n, *kernels in cases.LONG:
        got = choose([(d, d, g, 0, rows, k, n) for d in ("bf16", "fp32") for g in (False, True)])
        also = choose([("fp16", "fp16", g, 0, rows, k, n) for g in (False, True)])
        assert also == got[:2]
        for have, want in zip(got, kernels):
            assert want is None or have == want, (rows, k, n)


def test_every_large_kernel_is_reached():
    """Both forms of every type for which it is built, dense and per expert."""
    seen = {(c[-1][:3], c[0], c[1], "dense") for c in cases.DENSE}
    seen |= {(c[-1][:3], c[0], c[2], "grouped") for c in cases.GROUPED}
    for gated in (False, True):
        for dtype in ("bf16", "fp16"):
            assert (("tile", 8, 8), dtype, gated, "dense") in seen
            assert (("tile", 8, 8), dtype, gated, "grouped") in seen
        for form in ("dense", "grouped"):
            assert (("tile", 4, 4), "fp32", gated, form) in seen
        assert (("any", 2, 2), "fp32", gated, "dense") in seen
