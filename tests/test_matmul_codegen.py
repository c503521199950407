"""The 256 x 256 tile keeps its accumulators where inline matrix instructions put them.

The compiler knows nothing of the waits between such an instruction and a move of its
accumulator, so a move among them would give wrong results now and then.  This compiles
the kernel as the build does and looks at the assembly: between matrix instructions
there is no move of an accumulation register and no spill, and the waits stand behind
the last one."""

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
                        os.path.join(build.CSRC, "matmul_tile.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels = re.split(r"\n(?=_ZN3moe\w+:)", open(out).read())[1:]
    seen = 0
    for k in kernels:
        if "ELi8ELi8E" not in k.split(":")[0]:
            continue
        seen += 1
        code = [line.split(";")[0].strip() for line in k.split("\n")]
        mfma = [i for i, line in enumerate(code) if line.startswith("v_mfma")]
        assert len(mfma) == 3 * 256, "two steps in each of three straight blocks"
        written = [i for i, line in enumerate(code) if line.startswith("v_accvgpr")]
        assert not [i for i in written if mfma[0] < i < mfma[-1]], "an accumulator is moved between the steps"
        assert not [line for line in code[mfma[0]:mfma[-1]] if line.startswith("scratch_")], "a spill between the steps"
        # no vector instruction writes a register that a matrix instruction just behind it reads
        code = [line for line in code if line]
        for i, line in enumerate(code):
            m = re.match(r"v_(?!mfma|cmp|readfirst|readlane)\w+\s+v(?:\[(\d+):(\d+)\]|(\d+))", line)
            if not m:
                continue
            lo, hi = (int(m[1]), int(m[2])) if m[1] else (int(m[3]), int(m[3]))
            for near in code[i + 1:i + 5]:
                if near.startswith("v_mfma"):
                    for f, t in re.findall(r"v\[(\d+):(\d+)\]", near):
                        assert hi < int(f) or lo > int(t), f"{line} then {near}"
        mfma = [i for i, line in enumerate(code) if line.startswith("v_mfma")]
        written = [i for i, line in enumerate(code) if line.startswith("v_accvgpr")]
        after = [i for i in written if i > mfma[-1]]
        waits = [i for i, line in enumerate(code) if line == "s_nop 15" and i > mfma[-1]]
        assert len(waits) >= 2 and after and waits[1] < after[0], "the accumulators are read before the waits"
    assert seen == 4, "bf16 and fp16, plain and gated"
