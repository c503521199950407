"""The 128 x 128 tile of the integer products (and the 256 x 256 one, from the same source) rounds a value in the
same steps wherever it stands: its code holds none of the instructions that round a fused multiply-add straight
to fp16, which the compiler takes in some places of a tile and not in others."""

import os
import re
import subprocess

import pytest

from quantized_expert_gemv_moe_amd import build


def test_fp16_outputs_are_rounded_from_fp32(tmp_path):
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = str(tmp_path / "tile.s")
    r = subprocess.run([cc, *build._flags(), "-S", "--cuda-device-only", os.path.join(build.CSRC, "matmul_int_tile4.hip"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    code = open(out).read()
    assert re.search(r"v_cvt_pk_f16_f32|v_cvt_f16_f32", code)
    assert not re.search(r"v_(fma|mad)_mix(lo|hi)_f16", code)
