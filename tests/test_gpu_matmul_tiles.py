"""The products' kernels for large batches at shapes that reach them (matmul_cases.py, held to
the rule by test_matmul_choice.py), against the definitions in 64 bits."""

import numpy as np
import pytest
import torch

import matmul_cases as cases
import matmul_ref as ref
import quantized_expert_gemv_moe_amd as moe
from gpu_helpers import log
from test_gpu_matmul import check_grouped, gen, make_linear, name, normal, out_view, plan_of, reference, routing

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = {"bf16": BF16, "fp16": F16, "fp32": F32}


def ident(case):
    return "-".join(str(v) for v in case[:-1])


# function, bias, clamp, residual type (0: out's), out type (0: the weights')
FORMS = [("none", True, 0.0, 0, 0), ("silu", False, 0.0, None, 0), ("gelu", True, 0.9, F32, 0),
         ("gelu_tanh", True, 1.2, 0, F32), ("relu", False, 0.0, F16, BF16)]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f[0])
@pytest.mark.parametrize("case", cases.DENSE, ids=ident)
def test_dense(case, form):
    dtype, gated, rows, K, N, _ = case
    act, bias, clamp, res_dtype, out_dtype = form
    log(f"[case] dense {case} {form}")
    g = gen(rows + K + N)
    dt = TYPES[dtype]
    od = out_dtype or dt
    lin = make_linear(g, None, N, K, dt, gated, bias, act, od, clamp)
    x = normal(g, (rows, K), dt)
    res = None if res_dtype is None else normal(g, (rows, N), res_dtype or od)
    out, untouched = out_view(rows, N, od, 0)
    moe.matmul(lin, x, residual=res, out=out)
    again = moe.matmul(lin, x, residual=res)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, act, clamp, x, res), name(case=case, form=form))
    assert torch.equal(out, again)
    untouched()


@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("case", cases.GROUPED, ids=ident)
def test_grouped(case, rows):
    """With slots that no expert has, whose rows stay, and biases of the experts' own."""
    dtype, out_dtype, gated, E, T, k, K, N, _ = case
    rng = np.random.default_rng(T + K)
    idx = routing(rng, T, E, k, 0.6)
    idx[rng.random(idx.shape) < 0.02] = E
    idx[0, 0] = -1
    for act, bias, clamp in (("silu", False, 0.0), ("gelu", True, 0.9)):
        log(f"[case] grouped {case} rows={rows} {act}")
        check_grouped(idx, E, K, N, TYPES[dtype], gated, bias, act, TYPES[out_dtype], rows, clamp=clamp,
                      tag=name(case=case, rows=rows, act=act))


@pytest.mark.parametrize("case", [c for c in cases.GROUPED if c[-1] == cases.BIG], ids=ident)
def test_grouped_uneven(case):
    """Experts of one row and of a tile's rows and one more; an expert without rows."""
    dtype, out_dtype, gated, E, T, k, K, N, _ = case
    log(f"[case] grouped uneven {case}")
    flat = np.full(T * k, E - 1, np.int32)
    flat[T // 2] = 0
    if E > 3:
        flat[7:7 + 257] = 2  # and expert 1 has none
    check_grouped(flat.reshape(T, k), E, K, N, TYPES[dtype], gated, False, "silu", TYPES[out_dtype], "slot",
                  tag=name(case=case))


def far_rows(g, rows, cols, stride):
    """[rows, cols] bf16 rows `stride` elements apart, NaN just before and behind each."""
    buf = torch.empty((rows, stride), dtype=BF16, device="cuda")
    buf[:, cols:cols + 64] = float("nan")
    buf[:, -64:] = float("nan")
    v = buf[:, :cols]
    v.copy_(normal(g, (rows, cols), BF16))
    return v


def test_rows_of_x_near_16_mib_apart():
    """A tile of 256 rows of x whose offsets reach 4 GiB."""
    rows, K, N, stride, _ = cases.FAR_X
    log("[case] far rows of x")
    g = gen(51)
    lin = make_linear(g, None, N, K, BF16, False, False, "none", BF16)
    x = far_rows(g, rows, K, stride)
    out = moe.matmul(lin, x)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "none", 0.0, x), "far x")


def test_rows_of_w_near_16_mib_apart():
    rows, K, N, stride, _ = cases.FAR_W
    log("[case] far rows of w")
    g = gen(52)
    w = far_rows(g, N, K, stride)
    w.mul_(0.9 / K ** 0.5)
    lin = moe.Linear.from_tensors(w)
    x = normal(g, (rows, K), BF16)
    out = moe.matmul(lin, x)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "none", 0.0, x), "far w")


@pytest.mark.parametrize("rows", ["token", "slot"])
@pytest.mark.parametrize("case", cases.FAR_GATHERED, ids=ident)
def test_gathered_rows_just_below_4_gib(case, rows):
    E, n, K, N, stride, _ = case
    log(f"[case] far gathered {case} rows={rows}")
    g = gen(53)
    lin = make_linear(g, E, N, K, BF16, False, False, "none", BF16)
    idx, plan = plan_of(routing(np.random.default_rng(n), n, E, 1), E)
    x = far_rows(g, n, K, stride)
    out = moe.grouped_matmul(lin, x, plan, n, top_k=1, rows=rows)
    torch.cuda.synchronize()
    for e in range(E):
        mine = torch.nonzero(idx[:, 0] == e)[:, 0]
        ref.check(out[mine], *ref.product(x[mine], lin.w[e], out_dtype=BF16), f"{case} e={e}")


def test_functions_where_their_factor_underflows():
    """Far below zero f(z) = z times a factor below the normal range, which may count as zero;
    nothing else is lost on the way there."""
    log("[case] functions below -40")
    z = torch.linspace(-140, -6, 4001, device="cuda")
    x = z[:, None].contiguous()
    w = torch.ones((1, 1), device="cuda")
    for act in ("silu", "gelu", "gelu_tanh"):
        out = moe.matmul(moe.Linear.from_tensors(w, activation=act), x)
        torch.cuda.synchronize()
        want, tol = ref.product(x, w, act=act)
        ref.check(out, want, tol + z.double().abs()[:, None] * 2.0 ** -126, act)
