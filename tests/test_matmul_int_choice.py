"""Which kernel the library takes for the shapes of the integer products' GPU tests (CPU only: the rule is
host code).  A rule that is fitted anew may change these; the tests' shapes then have to follow, so
that every kernel stays tested."""

import os
import shutil
import subprocess

import pytest

import int_cases

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
DTYPES = {"fp32": 0, "bf16": 1, "fp16": 2, "int8": 3}


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("no C++ compiler or HIP headers")
    csrc = os.path.join(ROOT, "quantized_expert_gemv_moe_amd", "csrc")
    exe = str(tmp_path_factory.mktemp("choice") / "choice")
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I",
                    os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "matmul_abi.cpp"),
                    os.path.join(csrc, "matmul_int_abi.cpp"), os.path.join(HERE, "matmul_int_choice.cpp"), "-o", exe],
                   check=True)

    def run(queries):
        """Kernels of (x dtype, out dtype, gated, experts or 0, rows, K, N, top_k, offset of x, workspace); rows
        of w end at a whole chunk, as LinearInt lays them out."""
        lines = []
        for x, o, g, e, r, k, n, top, off, ws in queries:
            off *= {"fp32": 4, "int8": 1}.get(x, 2)
            lines.append(f"{DTYPES[x]} {DTYPES[o]} {int(g)} {e} {r} {k} {n} {top} {off} {-k % 16} {ws}")
        out = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, check=True).stdout
        return [(w[0], *map(int, w[1:])) for w in (line.split() for line in out.strip().split("\n"))]

    return run


def test_shapes_reach_their_kernels(choose):
    for by_token in (True, False):  # rows by token and by slot have the same rule
        got = choose([(x, o, g, e, t * top, k, n, top if by_token else 1, off, ws)
                      for x, o, g, e, t, top, k, n, off, ws, _ in int_cases.CASES])
        bad = [(c, h) for c, h in zip(int_cases.CASES, got) if c[-1] != h]
        if by_token:  # fewer rows of x than slots: they may be too few to be copied
            bad = [(c, h) for c, h in bad if not (c[0] == "int8" and c[5] > 1 and c[4] < 256)]
        assert not bad


def test_every_kernel_is_reached():
    seen = {(c[-1][:3], c[2], c[3] > 0, c[-1][3] > 1) for c in int_cases.CASES}
    for gated in (False, True):
        for grouped in (False, True):
            for tile in ((1, 2), (2, 2), (2, 4)):
                for split in (False, True):
                    assert (("deep", *tile), gated, grouped, split) in seen
            assert (("tile", 4, 4), gated, grouped, False) in seen
            assert (("tile", 8, 8), gated, grouped, False) in seen
            assert (("any", 2, 2), gated, grouped, False) in seen
            assert (("int_few", 1, 4), gated, grouped, False) in seen
        for other in (("int_few", 1, 1), ("int_few", 1, 2), ("few", 1, 0), ("few", 2, 0)):
            assert (other, gated, False, False) in seen
    assert {c[0] for c in int_cases.CASES} == set(DTYPES) and {c[1] for c in int_cases.CASES} == {"bf16", "fp16", "fp32"}
