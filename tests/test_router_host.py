"""Host side of the scored router (no GPU): descriptor layout, argument checks.  Every call here
returns before anything is enqueued."""

import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import quantized_expert_gemv_moe_amd as moe
import router_ref
from quantized_expert_gemv_moe_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # aligned, never dereferenced by host validation
GIB = 1 << 30
I, U = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED

LAYOUT = r"""
#include <stddef.h>
#include <stdio.h>
#include "moe_decode.h"
#define F(f) printf("%s %zu\n", #f, offsetof(moe_router_t, f));
int main(void) {
    F(n_experts) F(top_k) F(score) F(n_groups) F(top_groups) F(group_score) F(renormalise) F(scale) F(bias)
    printf("sizeof %zu\n", sizeof(moe_router_t));
    printf("values %d %d %d %d %d\n", MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID, MOE_GROUP_MAX, MOE_GROUP_TOP2, MOE_MAX_GROUPS);
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
    fields = dict(line.split() for line in lines[:9])
    assert {f: getattr(_lib.RouterStruct, f).offset for f, _ in _lib.RouterStruct._fields_} == {
        k: int(v) for k, v in fields.items()}
    assert int(lines[9].split()[1]) == C.sizeof(_lib.RouterStruct)
    assert [int(v) for v in lines[10].split()[1:]] == [
        moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID, moe.MOE_GROUP_MAX, moe.MOE_GROUP_TOP2, _lib.MOE_MAX_GROUPS]


def router(**kw):
    st = _lib.RouterStruct(n_experts=256, top_k=8, score=1, n_groups=8, top_groups=4, group_score=1, renormalise=1,
                           scale=2.5, bias=FAKE)
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def check(**kw):
    return moe.lib().moe_router_check(C.byref(router(**kw)))


def test_router_check():
    assert check() == moe.MOE_OK
    for kw in (dict(bias=None), dict(score=0), dict(group_score=0), dict(renormalise=0), dict(scale=1e-30),
               dict(n_experts=1, top_k=1, n_groups=1, top_groups=1), dict(n_experts=1024, n_groups=64, top_groups=1),
               dict(top_k=16), dict(n_experts=30, n_groups=5, top_groups=2, top_k=12), dict(top_groups=8)):
        assert check(**kw) == moe.MOE_OK, kw
    for kw in (dict(n_experts=0), dict(n_experts=-256), dict(top_k=0), dict(n_groups=0), dict(n_groups=-8), dict(n_groups=7),
               dict(top_groups=0), dict(top_groups=9), dict(score=2), dict(score=-1), dict(group_score=2),
               dict(group_score=-1), dict(renormalise=2), dict(renormalise=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(bias=FAKE + 2),
               dict(n_experts=64, top_groups=1, top_k=9), dict(n_experts=4, n_groups=1, top_groups=1, top_k=5)):
        assert check(**kw) == I, kw
    for kw in (dict(n_experts=1025, n_groups=1, top_groups=1), dict(top_k=17), dict(n_experts=1024, n_groups=128)):
        assert check(**kw) == U, kw
    assert moe.lib().moe_router_check(None) == I


def call(st=None, logits=FAKE + GIB, dtype=0, stride=0, T=4, idx=FAKE + 2 * GIB, w=FAKE + 3 * GIB, plan=None):
    st = router() if st is None else st
    if plan is None:
        return moe.lib().moe_router_topk(C.byref(st), logits, dtype, stride, T, idx, w, None)
    return moe.lib().moe_router_plan(C.byref(st), logits, dtype, stride, T, idx, w, C.byref(plan), None)


def test_router_refusals():
    good = _lib.PlanStruct(*[FAKE + (8 + i) * GIB for i in range(6)])
    assert call(T=0) == moe.MOE_OK
    out = 4 * 8 * 4
    for plan in (None, good):
        for kw in (dict(T=-1), dict(dtype=3), dict(dtype=-1), dict(stride=-1), dict(stride=255), dict(logits=None),
                   dict(idx=None), dict(w=None), dict(logits=FAKE + 2), dict(logits=FAKE + 1, dtype=1),
                   dict(idx=FAKE + 2), dict(w=FAKE + 1), dict(st=router(top_k=0)),
                   # outputs over one another, the logits, the bias
                   dict(idx=FAKE + 3 * GIB), dict(idx=FAKE + 3 * GIB + out - 4), dict(idx=FAKE + GIB),
                   dict(w=FAKE + GIB + 4 * 256 * 4 - 4), dict(idx=FAKE), dict(w=FAKE + 255 * 4),
                   dict(idx=FAKE + GIB + 2 * 300 * 4, stride=300)):
            assert call(plan=plan, **kw) == I, kw
        assert call(plan=plan, T=1 << 30) == U
        assert call(plan=plan, stride=(1 << 32) + 1) == U
    for i in (0, 1, 2, 3, 4, 5):
        bad = _lib.PlanStruct(*[None if j == i else FAKE + (8 + j) * GIB for j in range(6)])
        assert call(plan=bad) == I, i
    bad = _lib.PlanStruct(*[FAKE + (8 + i) * GIB + (8 if i == 5 else 0) for i in range(6)])
    assert call(plan=bad) == I


def test_every_shape_has_lanes_for_its_groups():
    """The kernels' division of a wave, as router_per_lane and router_four_lanes make it."""
    def lanes(E, G):
        per, p = E // G, 1
        while p < 32 and -(-per // p) * G > 64:
            p *= 2
        return p, -(-per // p) * G

    for E in range(1, 1025):
        for G in range(1, 65):
            if E % G == 0:
                p, n = lanes(E, G)
                assert n <= 64 and (G > 1 or p <= 16), (E, G)


def test_wrappers_refuse_without_a_device():
    for kw in (dict(score="tanh"), dict(group_score="sum"), dict(n_experts=2 ** 32 + 8), dict(top_k=2 ** 32 + 1),
               dict(bias=torch.zeros(8)), dict(bias=torch.zeros(9))):
        with pytest.raises(ValueError):
            moe.Router(**{**dict(n_experts=8, top_k=2), **kw})
    with pytest.raises(moe.MoeError):
        moe.Router(8, 9)
    with pytest.raises(ValueError):
        moe.router_topk(moe.Router(8, 2), torch.zeros((3, 8)))
    with pytest.raises(ValueError):
        moe.router_plan(moe.Router(8, 2), torch.zeros((3, 8)))


# the definition used by the GPU tests, at points that can be told by hand
def test_reference_plain_cases():
    l = np.array([[0.0, 2.0, 1.0, 2.0]])
    ids, w, _ = router_ref.route(l, "fp32", 2, "softmax")
    assert ids.tolist() == [[1, 3]] and np.allclose(w, 0.5)
    ids, w, _ = router_ref.route(l, "fp32", 2, "sigmoid", bias=[1.0, 0, 0, 0], renormalise=False, scale=2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1.0, 2 / (1 + np.exp(-2.0))]])
    # the group of the two middling experts beats that of the best one
    l = np.array([[3.0, -3.0, 2.0, 2.0]])
    assert router_ref.route(l, "fp32", 2, "sigmoid", n_groups=2, top_groups=1, by="top2")[0].tolist() == [[2, 3]]
    assert router_ref.route(l, "fp32", 2, "sigmoid", n_groups=2, top_groups=1, by="max")[0].tolist() == [[0, 1]]
    l = np.array([[-np.inf, 1.0, -np.inf, router_ref.LOWEST["fp32"]], [-np.inf] * 4, [0, np.nan, 0, 0]])
    ids, w, _ = router_ref.route(l, "fp32", 3, "softmax")
    assert ids.tolist() == [[1, 0, 2], [0, 1, 2], [-1, -1, -1]]
    assert w[:2].tolist() == [[1, 0, 0], [0, 0, 0]] and np.isnan(w[2]).all()
