"""Host side of the unquantised products (no GPU): descriptor layout, argument
checks, workspace sizes.  Every call here returns before anything is enqueued."""

import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

import quantized_expert_gemv_moe_amd as moe
from quantized_expert_gemv_moe_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # aligned, never dereferenced by host validation
GIB = 1 << 30


def linear(**kw):
    st = _lib.LinearStruct(in_features=2048, out_features=768, n_groups=1, dtype=moe.MOE_DTYPE_BF16,
                           out_dtype=moe.MOE_DTYPE_BF16, fn=moe.MOE_FN_SILU, clamp_limit=0.0, w=FAKE)
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def check(**kw):
    return moe.lib().moe_linear_check(C.byref(linear(**kw)))


LAYOUT = r"""
#include <stddef.h>
#include <stdio.h>
#include "moe_decode.h"
#define F(f) printf("%s %zu\n", #f, offsetof(moe_linear_t, f));
int main(void) {
    F(in_features) F(out_features) F(n_groups) F(dtype) F(out_dtype) F(fn) F(clamp_limit) F(reserved) F(w) F(w_up)
    F(bias) F(bias_up) F(row_stride) F(group_stride) F(bias_stride)
    printf("sizeof %zu\n", sizeof(moe_linear_t));
    printf("values %d %d %d %d %d %d %d %d %d\n", MOE_DTYPE_F16, MOE_FN_NONE, MOE_FN_RELU, MOE_FN_SILU, MOE_FN_GELU,
           MOE_FN_GELU_TANH, MOE_ROWS_TOKEN, MOE_ROWS_SLOT, MOE_ROWS_SORTED);
    return 0;
}
"""


def test_struct_and_constants_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "layout.c").write_text(LAYOUT)
    exe = str(tmp_path / "layout")
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(tmp_path / "layout.c"), "-o", exe], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    fields = dict(line.split() for line in lines[:15])
    assert {f: getattr(_lib.LinearStruct, f).offset for f, _ in _lib.LinearStruct._fields_} == {
        k: int(v) for k, v in fields.items()}
    assert int(lines[15].split()[1]) == C.sizeof(_lib.LinearStruct)
    assert [int(v) for v in lines[16].split()[1:]] == [
        moe.MOE_DTYPE_F16, moe.MOE_FN_NONE, moe.MOE_FN_RELU, moe.MOE_FN_SILU, moe.MOE_FN_GELU, moe.MOE_FN_GELU_TANH,
        moe.MOE_ROWS_TOKEN, moe.MOE_ROWS_SLOT, moe.MOE_ROWS_SORTED]


def test_linear_check_accepts():
    assert check() == moe.MOE_OK
    for d in range(3):
        for o in range(3):
            assert check(dtype=d, out_dtype=o) == moe.MOE_OK
    for fn in range(5):
        assert check(fn=fn) == moe.MOE_OK
    assert check(in_features=1, out_features=1) == moe.MOE_OK
    assert check(in_features=1003, out_features=1357, w=FAKE + 2) == moe.MOE_OK
    assert check(w_up=FAKE + GIB, bias=FAKE + 2 * GIB, bias_up=FAKE + 3 * GIB) == moe.MOE_OK
    assert check(w_up=FAKE + GIB) == moe.MOE_OK
    assert check(n_groups=1024, group_stride=2 * 768 * 2048, bias_stride=4096, bias=FAKE + 8 * GIB) == moe.MOE_OK
    assert check(row_stride=2051, clamp_limit=10.0) == moe.MOE_OK


@pytest.mark.parametrize("kw,want", [
    (dict(in_features=0), 1), (dict(out_features=0), 1), (dict(n_groups=0), 1), (dict(in_features=-5), 1),
    (dict(dtype=3), 1), (dict(out_dtype=-1), 1), (dict(fn=5), 1), (dict(fn=-1), 1), (dict(reserved=1), 1),
    (dict(clamp_limit=-1.0), 1), (dict(clamp_limit=float("nan")), 1), (dict(clamp_limit=float("inf")), 1),
    (dict(w=None), 1), (dict(w=FAKE + 1), 1), (dict(dtype=0, w=FAKE + 2), 1), (dict(w_up=FAKE + 1), 1),
    (dict(bias=FAKE + 1), 1), (dict(bias_up=FAKE), 1), (dict(w_up=FAKE + GIB, bias=FAKE), 1),
    (dict(bias=FAKE + GIB, bias_up=FAKE), 1),
    (dict(row_stride=-1), 1), (dict(row_stride=2047), 1), (dict(group_stride=-1), 1), (dict(bias_stride=-1), 1),
    (dict(n_groups=4, group_stride=768 * 2048 - 1), 1), (dict(n_groups=4, bias=FAKE, bias_stride=767), 1),
    (dict(n_groups=1025), 2), (dict(row_stride=1 << 23), 2), (dict(in_features=1 << 23), 2),
    (dict(dtype=0, in_features=1 << 22), 2), (dict(n_groups=2, group_stride=1 << 50), 2),
    (dict(n_groups=2, out_features=(1 << 31) - 1, in_features=1 << 20), 2)])
def test_linear_check_rejects(kw, want):
    assert check(**kw) == want


def call(lin=None, x=FAKE + GIB, xs=0, rows=8, res=None, rd=1, rs=0, out=FAKE + 2 * GIB, os_=0, ws=FAKE + 16 * GIB,
         wb=4 * GIB):
    lin = linear() if lin is None else lin
    return moe.lib().moe_matmul(C.byref(lin), x, xs, rows, res, rd, rs, out, os_, ws, wb, None)


def test_matmul_refusals():
    I, U = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert call(rows=0) == moe.MOE_OK  # nothing to launch
    assert moe.lib().moe_matmul(None, FAKE, 0, 0, None, 0, 0, FAKE, 0, None, 0, None) == I
    for kw in (dict(rows=-1), dict(x=None), dict(out=None), dict(x=FAKE + GIB + 1), dict(out=FAKE + 2 * GIB + 1),
               dict(xs=-1), dict(xs=2047), dict(os_=767), dict(os_=-768), dict(res=FAKE + 3 * GIB, rd=7),
               dict(res=FAKE + 3 * GIB + 1), dict(res=FAKE + 3 * GIB, rs=5), dict(res=FAKE + 3 * GIB, rs=-1),
               dict(lin=linear(n_groups=2)), dict(lin=linear(w=None))):
        assert call(**kw) == I, kw
    assert call(rows=1 << 30) == U
    assert call(xs=1 << 23) == U
    assert call(os_=1 << 23) == U
    # out over anything the call reads
    row_x, row_o = 2048 * 2, 768 * 2
    for out in (FAKE, FAKE + 768 * row_x - 2, FAKE + GIB, FAKE + GIB + 8 * row_x - 2, FAKE + GIB - 8 * row_o + 2):
        assert call(out=out) == I, hex(out)
    res = FAKE + 3 * GIB
    assert call(out=res + 2, res=res) == I
    assert call(out=res, res=res, rd=moe.MOE_DTYPE_F16) == I  # same place, another type
    assert call(out=res, res=res, rs=800) == I                 # same place, another stride
    b = FAKE + 4 * GIB
    assert call(lin=linear(bias=b), out=b) == I
    # two column ranges of one buffer that meet
    assert call(x=FAKE + GIB, xs=4096, out=FAKE + GIB + 2 * 2047, os_=4096) == I


def test_columns_of_one_buffer_do_not_overlap():
    """The same rule as a pure function of the spans, over all small layouts."""
    cells = {}
    for stride in (6, 8):
        for wa in (2, 3, 6):
            for wb in (1, 3, 5):
                for off in range(-14, 15):
                    for ra, rb in ((1, 1), (3, 1), (2, 4)):
                        a = {100 + i * stride + j for i in range(ra) for j in range(wa)}
                        b = {100 + off + i * stride + j for i in range(rb) for j in range(wb)}
                        cells[(stride, wa, wb, off, ra, rb)] = bool(a & b)
    # through the ABI: fp16 x of wa columns, out of wb columns, byte layouts scaled by 2
    base = FAKE + GIB
    for (stride, wa, wb, off, ra, rb), hit in cells.items():
        if ra != rb:
            continue
        lin = linear(in_features=wa, out_features=wb, dtype=2, out_dtype=2)
        if stride < max(wa, wb):
            continue
        got = moe.lib().moe_matmul(C.byref(lin), base, stride, -1 if not hit else ra, None, 0, 0, base + 2 * off,
                                   stride, None, 0, None)
        assert got == moe.MOE_ERR_INVALID_ARG  # overlap refused; the others stop at the negative row count


def gcall(lin=None, x=FAKE + GIB, xs=0, slots=64, k=8, rows=0, plan=True, out=FAKE + 2 * GIB, os_=0, work=FAKE + 3 * GIB,
          sorted_slots=FAKE + 4 * GIB):
    lin = linear(n_groups=128) if lin is None else lin
    p = _lib.PlanStruct(FAKE, FAKE, sorted_slots, FAKE, FAKE, work)
    return moe.lib().moe_grouped_matmul(C.byref(lin), x, xs, slots, k, rows, C.byref(p) if plan else None, out, os_,
                                        FAKE + 16 * GIB, 4 * GIB, None)


def test_grouped_refusals():
    I, U = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
    assert gcall(slots=0) == moe.MOE_OK
    for kw in (dict(slots=-1), dict(k=0), dict(rows=3), dict(rows=-1), dict(plan=False), dict(work=None),
               dict(work=FAKE + 8), dict(sorted_slots=None), dict(sorted_slots=None, rows=1), dict(x=None),
               dict(out=None), dict(out=FAKE), dict(out=FAKE + 127 * 768 * 2048 * 2), dict(out=FAKE + GIB),
               dict(xs=5), dict(os_=5)):
        assert gcall(**kw) == I, kw
    assert gcall(slots=1 << 30) == U


def test_workspace_must_not_overlap_the_plan():
    lin = linear(in_features=8192, out_features=512, n_groups=1)  # K goes in stretches
    need = moe.lib().moe_grouped_workspace_size(C.byref(lin), 16)
    ws = FAKE + 16 * GIB
    assert 0 < need <= 4 * GIB
    for kw in (dict(work=ws), dict(work=ws + 1024), dict(sorted_slots=ws + 256), dict(work=ws, rows=2)):
        assert gcall(lin=lin, slots=16, **kw) == moe.MOE_ERR_INVALID_ARG, kw


def test_combine_refusals():
    I, U = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED

    def combine(y=FAKE, yd=0, idx=FAKE + GIB, w=FAKE + 2 * GIB, T=4, H=64, k=2, E=8, res=None, rd=0, out=FAKE + 3 * GIB,
                od=0):
        return moe.lib().moe_combine(y, yd, idx, w, T, H, k, E, res, rd, out, od, None)

    assert combine(T=0) == moe.MOE_OK
    for kw in (dict(T=-1), dict(H=0), dict(k=0), dict(E=0), dict(yd=3), dict(od=-1), dict(res=FAKE + 4 * GIB, rd=9),
               dict(y=None), dict(idx=None), dict(w=None), dict(out=None), dict(y=FAKE + 2), dict(idx=FAKE + 2),
               dict(w=FAKE + 1), dict(out=FAKE + 2), dict(res=FAKE + 1), dict(out=FAKE), dict(out=FAKE + 2 * 4 * 64 * 4 - 4),
               dict(out=FAKE + GIB), dict(out=FAKE + 2 * GIB), dict(res=FAKE + 3 * GIB + 4),
               dict(res=FAKE + 3 * GIB, rd=1)):
        assert combine(**kw) == I, kw
    for kw in (dict(k=17, E=32), dict(E=1025), dict(H=1 << 22), dict(T=(1 << 30) - 1), dict(T=1 << 20, H=1 << 16)):
        assert combine(**kw) == U, kw


def test_workspace_sizes():
    L = moe.lib()
    for rows in (0, -1):
        assert L.moe_matmul_workspace_size(C.byref(linear()), rows) == 0
        assert L.moe_grouped_workspace_size(C.byref(linear(n_groups=8)), rows) == 0
    assert L.moe_matmul_workspace_size(C.byref(linear(w=None)), 8) == 0
    # the size for up to n rows serves every smaller batch
    for kw in (dict(), dict(in_features=8192, out_features=512), dict(dtype=0, w_up=FAKE + GIB), dict(in_features=1003)):
        last = 0
        for rows in list(range(1, 300)) + [512, 1000, 4096, 70000]:
            n = L.moe_matmul_workspace_size(C.byref(linear(**kw)), rows)
            assert n >= last, (kw, rows)
            last = n


def test_binding_refuses_host_tensors_and_bad_descriptors():
    w = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.Linear.from_tensors(w)
    with pytest.raises(ValueError):
        moe.Linear.from_tensors(w, activation="swish")
    with pytest.raises(ValueError):
        moe.combine(torch.zeros((4, 8)), torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)), 4)
