"""Host side of the 8-bit integer products and of the quantisation of rows (no GPU): descriptor
layout, argument checks, workspace sizes.  Every call here returns before anything is enqueued."""

import ctypes as C
import os
import shutil
import subprocess
from fractions import Fraction

import pytest
import torch

import int_ref
import quantized_expert_gemv_moe_amd as moe
from quantized_expert_gemv_moe_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # aligned, never dereferenced by host validation
GIB = 1 << 30
I, U, W = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE

LAYOUT = r"""
#include <stddef.h>
#include <stdio.h>
#include "moe_decode.h"
#define F(f) printf("%s %zu\n", #f, offsetof(moe_linear_int_t, f));
int main(void) {
    F(in_features) F(out_features) F(n_groups) F(out_dtype) F(fn) F(clamp_limit) F(bias_dtype) F(row_tail) F(w) F(w_up)
    F(w_scale) F(w_up_scale) F(bias) F(bias_up) F(row_stride) F(group_stride) F(scale_stride) F(bias_stride)
    printf("sizeof %zu\n", sizeof(moe_linear_int_t));
    printf("values %d %d\n", MOE_DTYPE_I8, MOE_MAX_I8_INPUTS);
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
    fields = dict(line.split() for line in lines[:18])
    assert {f: getattr(_lib.LinearIntStruct, f).offset for f, _ in _lib.LinearIntStruct._fields_} == {
        k: int(v) for k, v in fields.items()}
    assert int(lines[18].split()[1]) == C.sizeof(_lib.LinearIntStruct)
    assert [int(v) for v in lines[19].split()[1:]] == [moe.MOE_DTYPE_I8, _lib.MOE_MAX_I8_INPUTS]


def linear(**kw):
    st = _lib.LinearIntStruct(in_features=2048, out_features=768, n_groups=1, out_dtype=moe.MOE_DTYPE_BF16,
                              fn=moe.MOE_FN_SILU, w=FAKE, w_scale=FAKE + 4 * GIB)
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def check(**kw):
    return moe.lib().moe_linear_int_check(C.byref(linear(**kw)))


def test_linear_int_check():
    up = dict(w_up=FAKE + GIB, w_up_scale=FAKE + 5 * GIB)
    for kw in (dict(), up, dict(bias=FAKE), dict(bias=FAKE, bias_up=FAKE, **up), dict(w=FAKE + 1), dict(fn=4),
               dict(n_groups=1024, scale_stride=768, group_stride=768 * 2048), dict(in_features=131071, row_tail=1, row_stride=131072),
               dict(in_features=1003, row_tail=5, row_stride=1008), dict(out_dtype=0), dict(bias_dtype=2, bias=FAKE + 2),
               dict(clamp_limit=10.0), dict(in_features=1, out_features=1)):
        assert check(**kw) == moe.MOE_OK, kw
    for kw in (dict(in_features=0), dict(out_features=-1), dict(n_groups=0), dict(out_dtype=3), dict(bias_dtype=3),
               dict(out_dtype=-1), dict(fn=5), dict(fn=-1), dict(clamp_limit=-1.0), dict(clamp_limit=float("nan")),
               dict(w=None), dict(w_scale=None), dict(w_up=FAKE), dict(w_up_scale=FAKE), dict(bias_up=FAKE),
               dict(bias=FAKE, **up), dict(bias=FAKE, bias_up=FAKE), dict(bias_up=FAKE, **up), dict(w_scale=FAKE + 2),
               dict(bias=FAKE + 2), dict(bias_dtype=1, bias=FAKE + 1), dict(row_stride=-1), dict(row_stride=2047),
               dict(group_stride=-1), dict(scale_stride=-1), dict(bias_stride=-1), dict(row_tail=-1), dict(row_tail=16),
               dict(row_tail=1), dict(row_tail=8, row_stride=2050), dict(n_groups=2, group_stride=768 * 2048 - 1),
               dict(n_groups=2, scale_stride=767), dict(n_groups=2, bias=FAKE, bias_stride=5)):
        assert check(**kw) == I, kw
    for kw in (dict(n_groups=1025), dict(in_features=131072), dict(row_stride=1 << 24),
               dict(n_groups=2, group_stride=1 << 41), dict(n_groups=2, scale_stride=1 << 41)):
        assert check(**kw) == U, kw
    assert moe.lib().moe_linear_int_check(None) == I


WS, OUT, X, XS, RES = FAKE + 32 * GIB, FAKE + 16 * GIB, FAKE + 8 * GIB, FAKE + 12 * GIB, FAKE + 20 * GIB


def call(lin=None, x=X, xd=3, xs=0, scale=XS, rows=8, res=None, rd=1, rs=0, out=OUT, os_=0, ws=WS, wb=4 * GIB):
    lin = linear() if lin is None else lin
    if xd != 3 and scale == XS:
        scale = None
    return moe.lib().moe_matmul_int(C.byref(lin), x, xd, xs, scale, rows, res, rd, rs, out, os_, ws, wb, None)


def test_matmul_int_refusals():
    for xd in (0, 1, 3):
        assert call(rows=0, xd=xd) == moe.MOE_OK
        es = {0: 4, 1: 2, 3: 1}[xd]
        for kw in (dict(rows=-1), dict(x=None), dict(out=None), dict(xs=-1), dict(xs=2047), dict(os_=767), dict(os_=-768),
                   dict(out=OUT + 1), dict(res=RES, rd=7), dict(res=RES + 1), dict(res=RES, rs=5), dict(res=RES, rs=-1),
                   dict(lin=linear(n_groups=2)), dict(lin=linear(w=None)),
                   # out over what the call reads
                   dict(out=FAKE), dict(out=FAKE + 768 * 2048 - 2), dict(out=FAKE + 4 * GIB), dict(out=FAKE + 4 * GIB + 767 * 4),
                   dict(out=X), dict(out=X + 8 * 2048 * es - 2), dict(out=RES + 2, res=RES),
                   dict(out=RES, res=RES, rd=2), dict(out=RES, res=RES, rs=800),
                   dict(out=FAKE + 5 * GIB, lin=linear(w_up=FAKE + GIB, w_up_scale=FAKE + 5 * GIB)),
                   dict(out=FAKE + 6 * GIB, lin=linear(bias=FAKE + 6 * GIB))):
            assert call(xd=xd, **kw) == I, (xd, kw)
        assert call(xd=xd, rows=1 << 30) == U
        assert call(xd=xd, xs=1 << 24) == U
        assert call(xd=xd, os_=1 << 23) == U
    for kw in (dict(xd=4), dict(xd=-1), dict(xd=3, scale=None), dict(xd=3, scale=XS + 2), dict(xd=1, scale=XS + GIB),
               dict(xd=0, x=X + 2), dict(xd=1, x=X + 1), dict(xd=3, out=XS), dict(xd=3, out=XS + 28)):
        assert call(**kw) == I, kw


def test_matmul_int_workspace_checks():
    lin = linear()
    need = moe.lib().moe_matmul_int_workspace_size(C.byref(lin), 8)
    assert need >= 8 * 2048 + 8 * 4
    for kw in (dict(ws=None), dict(ws=WS + 128), dict(ws=X), dict(ws=X + 8 * 2048 * 2 - 256 + 256 - 256), dict(ws=OUT),
               dict(ws=FAKE), dict(ws=FAKE + 4 * GIB), dict(ws=FAKE + 4 * GIB + 256), dict(ws=RES, res=RES)):
        assert call(xd=1, **kw) == I, kw
    assert call(xd=1, wb=8 * 2048) == W
    assert call(xd=1, wb=0) == W
    # few tiles over a long K: the product has a part of its own behind the integers
    lin = linear(in_features=65536, out_features=64)
    assert moe.lib().moe_matmul_int_workspace_size(C.byref(lin), 64) > 64 * 65536 + 256
    assert call(lin=lin, rows=64, xd=1, wb=64 * 65536 + 256) == W


def gcall(lin=None, x=X, xd=3, xs=0, scale=XS, slots=64, k=8, rows=0, plan=True, out=OUT, os_=0, work=FAKE + 24 * GIB,
          sorted_slots=FAKE + 25 * GIB, ws=WS, wb=4 * GIB):
    lin = linear(n_groups=128) if lin is None else lin
    p = _lib.PlanStruct(FAKE, FAKE, sorted_slots, FAKE, FAKE, work)
    if xd != 3:
        scale = None
    return moe.lib().moe_grouped_matmul_int(C.byref(lin), x, xd, xs, scale, slots, k, rows, C.byref(p) if plan else None,
                                            out, os_, ws, wb, None)


def test_grouped_int_refusals():
    for xd in (0, 1, 3):
        assert gcall(slots=0, xd=xd) == moe.MOE_OK
        for kw in (dict(slots=-1), dict(k=0), dict(k=-2), dict(rows=3), dict(rows=-1), dict(plan=False), dict(work=None),
                   dict(work=FAKE + 8), dict(sorted_slots=None), dict(sorted_slots=None, rows=1), dict(x=None),
                   dict(out=None), dict(out=FAKE), dict(out=FAKE + 127 * 768 * 2048), dict(out=X), dict(xs=5), dict(os_=5),
                   dict(out=FAKE + 4 * GIB + 127 * 768 * 4), dict(out=FAKE + 24 * GIB), dict(out=FAKE + 25 * GIB)):
            assert gcall(xd=xd, **kw) == I, (xd, kw)
        assert gcall(slots=1 << 30, xd=xd) == U
    for kw in (dict(work=WS), dict(sorted_slots=WS + 256), dict(ws=X), dict(ws=FAKE + 100 * 768 * 2048),
               dict(ws=FAKE + 4 * GIB + 256)):
        assert gcall(xd=1, **kw) == I, kw
    assert gcall(xd=1, wb=8 * 2048) == W
    assert gcall(xd=1, rows=1, wb=63 * 2048) == W


def test_workspace_sizes():
    L = moe.lib()
    lin, bad = linear(n_groups=8), linear(w=None)
    for n in (0, -1):
        assert L.moe_matmul_int_workspace_size(C.byref(linear()), n) == 0
        assert L.moe_grouped_int_workspace_size(C.byref(lin), n, 4) == 0
        assert L.moe_grouped_int_workspace_size(C.byref(lin), 4, n) == 0
    assert L.moe_matmul_int_workspace_size(C.byref(bad), 8) == 0
    for kw in (dict(), dict(in_features=8192, out_features=512), dict(in_features=1003, row_stride=1008, row_tail=5)):
        last = 0
        for rows in list(range(1, 300)) + [512, 1000, 4096, 70000]:
            n = L.moe_matmul_int_workspace_size(C.byref(linear(**kw)), rows)
            assert n >= last and n % 256 == 0, (kw, rows)
            last = n


def quant(x=X, d=1, xs=0, rows=4, cols=100, codes=OUT, cs=0, scales=XS):
    return moe.lib().moe_quantize_rows(x, d, xs, rows, cols, codes, cs, scales, None)


def test_quantize_refusals():
    assert quant(rows=0) == moe.MOE_OK
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=-5), dict(d=3), dict(d=-1), dict(xs=-1), dict(xs=99), dict(cs=-1),
               dict(cs=99), dict(x=None), dict(codes=None), dict(scales=None), dict(x=X + 1), dict(d=0, x=X + 2),
               dict(scales=XS + 2), dict(codes=X), dict(codes=X + 799), dict(scales=X + 400), dict(codes=XS + 3),
               dict(codes=XS - 399)):
        assert quant(**kw) == I, kw
    for kw in (dict(rows=1 << 30), dict(xs=1 << 23), dict(cs=1 << 24), dict(d=0, xs=1 << 22)):
        assert quant(**kw) == U, kw


def test_reference_rounds_the_exact_quotient():
    g = torch.Generator().manual_seed(1)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x = torch.randn((6, 50), generator=g).to(dtype)
        x[1, :] = (torch.arange(50) - 25.0) / 2  # halves
        x[1, 0] = 127.0
        x[2, 3] = 0.25
        q, s = int_ref.quantize(x)
        for r in range(6):
            row = [Fraction(float(v)) for v in x[r]]
            m = max(abs(v) for v in row)
            assert [int(v) for v in q[r]] == [round(v * 127 / m) for v in row]  # Fraction rounds half to even
            assert float(s[r]) == float(torch.tensor(float(m), dtype=torch.float32) / 127.0)


def test_wrappers_refuse_without_a_device():
    w, s = torch.zeros((4, 16), dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError):
        moe.LinearInt.from_tensors(w, s)
    with pytest.raises(ValueError):
        moe.LinearInt.from_tensors(w, s, activation="swish")
    with pytest.raises(ValueError):
        moe.LinearInt.from_tensors(w, s, clamp_limit=1e-50)
    with pytest.raises(ValueError):
        moe.quantize_rows(torch.zeros((4, 16)))

    class Described:
        struct = linear()

    for rows in (2 ** 32 + 5, 2 ** 31):
        with pytest.raises(ValueError, match="32 bits"):
            moe.matmul_int_workspace_size(Described(), rows)
        with pytest.raises(ValueError, match="32 bits"):
            moe.grouped_int_workspace_size(Described(), 8, rows)
