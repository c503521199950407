"""The 256 x 256 tile of the integer products keeps its accumulators where inline matrix instructions put
them, as test_matmul_codegen looks at it for the 16-bit types: no move of an accumulation register and no
spill between matrix instructions, no operand written right ahead of them, and the waits behind the last
one."""

import os
import re
import subprocess

import pytest

from quantized_expert_gemv_moe_amd import build


def test_no_accumulator_moves_between_matrix_instructions(tmp_path):
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = str(tmp_path / "tile.s")
    r = subprocess.run([cc, *build._flags(), "-S", "--cuda-device-only",
                        os.path.join(build.CSRC, "matmul_int_tile.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = 0
    for k in re.split(r"\n(?=_ZN3moe\w+:)", open(out).read())[1:]:
        if "matmul_tile_kernelILi3E" not in k.split(":")[0]:
            continue
        seen += 1
        code = [c for c in (line.split(";")[0].strip() for line in k.split("\n")) if c]
        mfma = [i for i, line in enumerate(code) if line.startswith("v_mfma")]
        assert len(mfma) == 3 * 256, "two steps in each of three straight blocks"
        assert all("i32_16x16x64_i8" in code[i] for i in mfma)
        between = code[mfma[0]:mfma[-1]]
        assert not [c for c in between if c.startswith(("v_accvgpr", "scratch_"))], "an accumulator is moved between the steps"
        for i, line in enumerate(code):  # no vector instruction writes what a matrix instruction just behind it reads
            m = re.match(r"v_(?!mfma|cmp|readfirst|readlane)\w+\s+v(?:\[(\d+):(\d+)\]|(\d+))", line)
            if not m:
                continue
            lo, hi = (int(m[1]), int(m[2])) if m[1] else (int(m[3]), int(m[3]))
            for near in code[i + 1:i + 5]:
                if near.startswith("v_mfma"):
                    for f, t in re.findall(r"v\[(\d+):(\d+)\]", near):
                        assert hi < int(f) or lo > int(t), f"{line} then {near}"
        after = [i for i, line in enumerate(code) if line.startswith("v_accvgpr") and i > mfma[-1]]
        waits = [i for i, line in enumerate(code) if line == "s_nop 15" and i > mfma[-1]]
        assert len(waits) >= 2 and after and waits[1] < after[0], "the accumulators are read before the waits"
    assert seen == 2, "plain and gated"
