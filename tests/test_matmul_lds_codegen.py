"""Loads into LDS by inline assembly tell the compiler that they write m0.

A kernel of its own interleaves them with the compiler's own loads into LDS, whose
target also goes through m0: the compiler may keep a value there from one of its loads to
the next only if nothing between writes the register."""

import os
import subprocess

import pytest

from quantized_expert_gemv_moe_amd import build

KERNEL = r"""
#include "matmul_lds.h"

extern "C" __global__ void interleaved(const char *from, uint32_t at, unsigned off) {
    __shared__ char lds[4096];
    typedef __attribute__((address_space(1))) const void *Global;
    typedef __attribute__((address_space(3))) void *Local;
    const char *p = from + threadIdx.x * 16;
    __builtin_amdgcn_global_load_lds((Global)p, (Local)lds, 16, 0, 0);
    moe::dma16(at, FORM);
    __builtin_amdgcn_global_load_lds((Global)(p + 4096), (Local)lds, 16, 0, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    ((char *)from)[threadIdx.x] = lds[threadIdx.x + off];
}
"""


@pytest.mark.parametrize("form", ["from, threadIdx.x * 16u", "p"], ids=["base and offset", "address"])
def test_m0_is_set_again_behind_an_inline_load(tmp_path, form):
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    src, out = tmp_path / "interleaved.hip", tmp_path / "interleaved.s"
    src.write_text(KERNEL.replace("FORM", form))
    r = subprocess.run([cc, *build._flags(), "-S", "--cuda-device-only", str(src), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    code = [line.split(";")[0].strip() for line in out.read_text().split("\n")]
    loads = [i for i, line in enumerate(code) if line.startswith("global_load_lds_dwordx4")]
    assert len(loads) == 3
    writes = [i for i, line in enumerate(code) if line.startswith("s_mov_b32 m0")]
    for before, load in zip([0] + loads, loads):
        assert [i for i in writes if before < i < load], f"line {load} uses the m0 of an earlier load"
