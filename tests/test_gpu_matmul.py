"""moe_matmul, moe_grouped_matmul and moe_combine on the GPU against their
definitions in 64 bits (matmul_ref.py derives the tolerances)."""

import numpy as np
import pytest
import torch

import matmul_ref as ref
import quantized_expert_gemv_moe_amd as moe
from gpu_helpers import log

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 12345.0  # exact in fp32; 12352 in bf16, 12344 in fp16: compared as stored


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=F32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def strided(g, rows, cols, dtype, pad, std=1.0, offset=0):
    """[rows, cols] view of a wider NaN-filled buffer, `offset` elements in."""
    buf = torch.full((rows * (cols + pad) + offset + 64,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(normal(g, (rows, cols), dtype, std))
    return v


def out_view(rows, cols, dtype, pad, offset=0):
    """An out view inside a sentinel-filled buffer, and a check that only the view was written."""
    buf = torch.full((rows * (cols + pad) + offset + 64,), SENTINEL, dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    def untouched():
        mine = torch.zeros_like(buf, dtype=torch.bool)
        mine[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = True
        s = torch.tensor(SENTINEL, dtype=dtype, device="cuda")
        assert bool((buf[~mine] == s).all()), "wrote outside out"

    return v, untouched


def make_linear(g, E, N, K, dtype, gated, bias, act, out_dtype, clamp=0.0, w_pad=0):
    lead = () if E is None else (E,)
    std = 0.9 / K ** 0.5

    def mat():
        m = torch.full(lead + (N, K + w_pad), float("nan"), dtype=dtype, device="cuda")[..., :K]
        m.copy_(normal(g, lead + (N, K), dtype, std))
        return m

    w = mat()
    w_up = mat() if gated else None
    b = normal(g, lead + (N,), dtype, 0.5) if bias else None
    b_up = normal(g, lead + (N,), dtype, 0.5) if bias and gated else None
    return moe.Linear.from_tensors(w, bias=b, w_up=w_up, bias_up=b_up, activation=act, out_dtype=out_dtype,
                                   clamp_limit=clamp)


def reference(lin, act, clamp, x, residual=None, e=None):
    def pick(t):
        return t if t is None or e is None else t[e]

    return ref.product(x, pick(lin.w), pick(lin.bias), pick(lin.w_up), pick(lin.bias_up), act, clamp, residual,
                       lin.out_dtype)


def name(**kw):
    return " ".join(f"{k}={v}" for k, v in kw.items())


# ------------------------------------------------------------------ matmul
# rows, K, N: one token to long batches, every remainder of the tiles, chunks
# and steps, sizes below one chunk
SHAPES = [(1, 1, 1), (1, 8, 16), (1, 2048, 768), (2, 64, 64), (3, 7, 5), (5, 100, 33), (16, 768, 2048), (17, 72, 130),
          (31, 1003, 257), (33, 40, 48), (64, 64, 64), (65, 520, 65), (77, 1003, 1357), (128, 136, 96),
          (129, 2048, 129), (200, 4104, 72), (256, 256, 256), (300, 256, 500), (513, 333, 127), (700, 1024, 640),
          (1024, 2048, 768)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matmul_shapes(shape, gated, dtype):
    rows, K, N = shape
    log(f"[case] matmul {shape} gated={gated} {dtype}")
    g = gen(rows * 7 + K + N)
    lin = make_linear(g, None, N, K, dtype, gated, True, "silu", dtype)
    x = normal(g, (rows, K), dtype)
    res = normal(g, (rows, N), dtype)
    out, untouched = out_view(rows, N, dtype, 0)
    got = moe.matmul(lin, x, residual=res, out=out)
    torch.cuda.synchronize()
    assert got is out
    ref.check(out, *reference(lin, "silu", 0.0, x, res), name(shape=shape, gated=gated, dtype=dtype))
    untouched()


# few tiles over a long K: the inputs are split over workgroups through the workspace
LONG = [(1, 16384, 64), (20, 8192, 96), (64, 8192, 512), (100, 4104, 130), (200, 8192, 300), (300, 16392, 64)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_matmul_long_inputs(shape, gated, dtype):
    """With a workspace full of NaN, exactly as large as asked for and between sentinels; one too
    small is refused."""
    rows, K, N = shape
    log(f"[case] long {shape} gated={gated} {dtype}")
    g = gen(rows + K + N)
    lin = make_linear(g, None, N, K, dtype, gated, True, "silu", dtype)
    x, res = normal(g, (rows, K), dtype), normal(g, (rows, N), F32)
    need = moe.matmul_workspace_size(lin, rows)
    assert need > 0
    buf = torch.full((need // 4 + 128,), float("nan"), device="cuda")
    buf[:64], buf[-64:] = SENTINEL, SENTINEL
    ws = buf[64:-64]
    out, untouched = out_view(rows, N, dtype, 0)
    moe.matmul(lin, x, residual=res, out=out, workspace=ws)
    again = moe.matmul(lin, x, residual=res)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "silu", 0.0, x, res), name(shape=shape, gated=gated, dtype=dtype))
    assert torch.equal(out, again)
    assert bool((buf[:64] == SENTINEL).all()) and bool((buf[-64:] == SENTINEL).all()), "wrote outside the workspace"
    untouched()
    if torch.isnan(ws[0]):
        return  # this shape took a kernel without a workspace
    with pytest.raises(moe.MoeError) as e:
        moe.matmul(lin, x, residual=res, out=out, workspace=ws[:64])
    assert e.value.status == moe.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (3, 4, 2), (40, 3, 2), (100, 2, 1)])
def test_grouped_long_inputs(T, E, k, rows):
    idx = routing(np.random.default_rng(T), T, E, k)
    for dtype, gated in ((BF16, True), (F16, False), (F32, False)):
        log(f"[case] grouped long T={T} E={E} k={k} rows={rows} {dtype}")
        check_grouped(idx, E, 8192, 64, dtype, gated, True, "silu", dtype, rows, tag=name(T=T, rows=rows, dtype=dtype))


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("out_dtype", [BF16, F16, F32], ids=["obf16", "ofp16", "ofp32"])
@pytest.mark.parametrize("rows", [3, 70])
def test_matmul_functions_and_output_types(rows, out_dtype, act):
    log(f"[case] matmul act={act} out={out_dtype} rows={rows}")
    g = gen(11)
    for gated, clamp, res_dtype in ((False, 0.0, None), (True, 0.0, F32), (True, 0.75, BF16), (False, 1.5, F16)):
        lin = make_linear(g, None, 88, 192, BF16, gated, clamp > 0, act, out_dtype, clamp)
        x = normal(g, (rows, 192), BF16, 3.0)
        res = None if res_dtype is None else normal(g, (rows, 88), res_dtype)
        out = moe.matmul(lin, x, residual=res)
        torch.cuda.synchronize()
        assert out.dtype == out_dtype
        ref.check(out, *reference(lin, act, clamp, x, res), name(act=act, gated=gated, clamp=clamp))


def test_matmul_functions_far_from_zero():
    """f at large arguments of both signs, at zero and at infinities, fp32 out: one input of
    weight one, so z is the input itself."""
    z = torch.cat([torch.linspace(-40, 40, 4001, device="cuda"),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e38, float("inf"), float("nan")], device="cuda")])
    x = z[:, None].contiguous()
    w = torch.ones((1, 1), device="cuda")
    for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
        lin = moe.Linear.from_tensors(w, activation=act)
        out = moe.matmul(lin, x)
        torch.cuda.synchronize()
        want, tol = ref.product(x, w, act=act)
        ref.check(out, want, tol + 1e-37, act)  # results below the fp32 normal range may flush


@pytest.mark.parametrize("rows,K,N", [(1, 256, 48), (9, 128, 100), (40, 264, 72), (150, 512, 200), (300, 1024, 384)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_matmul_strides_and_offsets(rows, K, N, dtype):
    """Rows of x, w, residual and out apart and at every element offset; nothing
    outside the rows is read (NaN there) or written."""
    for x_pad, w_pad, o_pad, offset in ((0, 0, 0, 1), (8, 8, 4, 0), (3, 0, 1, 3), (0, 5, 2, 0), (64, 64, 64, 8)):
        log(f"[case] strides rows={rows} K={K} N={N} {dtype} pads={x_pad},{w_pad},{o_pad} offset={offset}")
        g = gen(rows + x_pad)
        lin = make_linear(g, None, N, K, dtype, True, True, "gelu_tanh", dtype, w_pad=w_pad)
        x = strided(g, rows, K, dtype, x_pad, offset=offset)
        res = strided(g, rows, N, F16, o_pad, offset=offset)
        out, untouched = out_view(rows, N, dtype, o_pad, offset=offset)
        moe.matmul(lin, x, residual=res, out=out)
        torch.cuda.synchronize()
        ref.check(out, *reference(lin, "gelu_tanh", 0.0, x, res), name(pads=(x_pad, w_pad, o_pad, offset)))
        untouched()


@pytest.mark.parametrize("rows", [2, 100, 600])
def test_matmul_halves_of_one_buffer(rows):
    """gate and up as halves of one weight stack, x and out as column halves of one buffer."""
    g = gen(5)
    N, K = 96, 320
    gu = normal(g, (2 * N, K), BF16, 0.05)
    lin = moe.Linear.from_tensors(gu[:N], w_up=gu[N:], activation="silu")
    buf = torch.full((rows, K + N), float("nan"), dtype=BF16, device="cuda")
    buf[:, :K] = normal(g, (rows, K), BF16)
    x = buf[:, :K].clone()
    moe.matmul(lin, buf[:, :K], out=buf[:, K:])
    torch.cuda.synchronize()
    ref.check(buf[:, K:], *reference(lin, "silu", 0.0, x), "halves")
    assert torch.equal(buf[:, :K], x)


@pytest.mark.parametrize("rows", [1, 50, 260])
def test_matmul_adds_onto_its_residual_in_place(rows):
    g = gen(6)
    lin = make_linear(g, None, 256, 128, BF16, False, False, "none", BF16)
    x, r = normal(g, (rows, 128), BF16), normal(g, (rows, 256), BF16)
    h = r.clone()
    moe.matmul(lin, x, residual=h, out=h)
    torch.cuda.synchronize()
    ref.check(h, *reference(lin, "none", 0.0, x, r), "in place")


@pytest.mark.parametrize("rows", [1, 8, 40, 140, 1000])
@pytest.mark.parametrize("K", [96, 1001])
def test_matmul_nan_and_inf_stay_in_their_row_and_column(rows, K):
    g = gen(8)
    N = 130
    lin = make_linear(g, None, N, K, BF16, False, False, "none", F32)
    x = normal(g, (rows, K), BF16)
    if rows > 1:
        x[rows // 2, K - 1] = float("nan")
    x[0, K // 2] = float("inf")
    lin.w[17, 0] = float("nan")
    out = moe.matmul(lin, x)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "none", 0.0, x), f"rows={rows} K={K}")


def test_matmul_overflow_and_small_values_fp16():
    g = gen(9)
    w = torch.ones((40, 64), dtype=F16, device="cuda")
    x = torch.full((20, 64), 2000.0, dtype=F16, device="cuda")
    x[1] = -2000.0
    x[2] = 6e-8  # a subnormal
    lin = moe.Linear.from_tensors(w)
    out = moe.matmul(lin, x)
    torch.cuda.synchronize()
    want, tol = reference(lin, "none", 0.0, x)
    assert bool(torch.isinf(out[0]).all()) and bool(torch.isinf(out[1]).all()) and bool((out[1] < 0).all())
    ref.check(out[2:], want[2:], tol[2:], "small values")


@pytest.mark.parametrize("rows,K,N", [(1, 4096, 512), (24, 2048, 512), (180, 2048, 1024), (2000, 512, 768)])
def test_matmul_is_reproducible_and_rows_keep_to_themselves(rows, K, N):
    """Twice the same bits; a row's neighbours (their values, not their number) change nothing."""
    g = gen(12)
    lin = make_linear(g, None, N, K, BF16, True, False, "silu", BF16)
    x = normal(g, (rows, K), BF16)
    a = moe.matmul(lin, x)
    b = moe.matmul(lin, x)
    y = normal(g, (rows, K), BF16)
    y[rows // 3] = x[rows // 3]
    c = moe.matmul(lin, y)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(a[rows // 3].view(torch.int16), c[rows // 3].view(torch.int16))


# sizes at which the large tiles run, with ends inside a tile and a step
LARGE = [(4096, 520, 4096), (4096, 512, 4000), (4100, 512, 4104), (2048, 2048, 2048), (3000, 4096, 1100)]
LARGE_FORMS = [  # gated, function, out type (None: the weights'), residual type (0: the weights'), clamp
    (False, "none", None, 0, 0.0), (False, "silu", None, None, 0.0), (False, "gelu_tanh", None, 0, 1.5),
    (False, "gelu", None, None, 0.0), (False, "relu", None, F32, 0.0), (False, "none", F32, F32, 0.0),
    (True, "silu", None, None, 0.0), (True, "gelu_tanh", None, 0, 0.8), (True, "silu", F32, None, 0.0)]


@pytest.mark.parametrize("form", LARGE_FORMS, ids=lambda f: "-".join(str(v).replace("torch.", "") for v in f))
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_matmul_large_tiles(shape, form):
    rows, K, N = shape
    gated, act, out_dtype, res_dtype, clamp = form
    for dtype in (BF16, F16):
        log(f"[case] large {shape} {form} {dtype}")
        g = gen(rows + K)
        od = out_dtype or dtype
        lin = make_linear(g, None, N, K, dtype, gated, True, act, od, clamp)
        x = normal(g, (rows, K), dtype)
        res = None if res_dtype is None else normal(g, (rows, N), res_dtype or dtype)
        out, untouched = out_view(rows, N, od, 0)
        moe.matmul(lin, x, residual=res, out=out)
        torch.cuda.synchronize()
        ref.check(out, *reference(lin, act, clamp, x, res), name(shape=shape, form=form, dtype=dtype))
        untouched()
        if res is not None and res.dtype == od:  # onto its residual, in place
            moe.matmul(lin, x, residual=res, out=res)
            torch.cuda.synchronize()
            assert torch.equal(res, out)


@pytest.mark.parametrize("pad,offset", [(4, 0), (8, 0), (0, 4), (1, 0), (0, 1)])
def test_matmul_large_tiles_into_strided_rows(pad, offset):
    g = gen(14)
    rows, K, N = 4096, 512, 4096
    lin = make_linear(g, None, N, K, BF16, False, False, "silu", BF16)
    x = normal(g, (rows, K), BF16)
    res = strided(g, rows, N, BF16, pad, offset=offset)
    out, untouched = out_view(rows, N, BF16, pad, offset=offset)
    moe.matmul(lin, x, residual=res, out=out)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "silu", 0.0, x, res), f"pad {pad} offset {offset}")
    untouched()


@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("T,E,k,K,N,gated", [(6000, 4, 2, 520, 2048, False), (6000, 4, 2, 512, 1000, True),
                                             (9000, 16, 2, 264, 1024, True), (5000, 3, 1, 2048, 2048, False)])
def test_grouped_large_tiles(T, E, k, K, N, gated, rows):
    rng = np.random.default_rng(T)
    idx = routing(rng, T, E, k, 0.7)
    idx[rng.random(idx.shape) < 0.02] = E
    for act, od, clamp in (("silu", BF16, 0.0), ("gelu", F32, 0.9)):
        log(f"[case] grouped large T={T} E={E} K={K} N={N} gated={gated} rows={rows} {act}")
        check_grouped(idx, E, K, N, BF16, gated, True, act, od, rows, clamp=clamp, tag=name(T=T, E=E, rows=rows, act=act))


def test_offsets_past_32_bits():
    """Rows of x and out spread over more than 4 GiB, in order and gathered through a plan."""
    g = gen(13)
    T, K, N, stride = 140000, 64, 40, 16384  # 32 KiB between rows: 4.6 GB
    xb = torch.empty((T, stride), dtype=BF16, device="cuda")
    x = xb[:, :K]
    x.copy_(normal(g, (T, K), BF16))
    ob = torch.empty((T, stride), dtype=BF16, device="cuda")
    out = ob[:, :N]
    lin = make_linear(g, None, N, K, BF16, False, True, "none", BF16)
    moe.matmul(lin, x, out=out)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "none", 0.0, x), "in order")
    el = make_linear(g, 2, N, K, BF16, False, False, "none", BF16)
    idx = (torch.arange(T, device="cuda") * 7 // 3 % 2).to(torch.int32).view(T, 1)
    plan = moe.expert_plan(idx, 2)
    for rows in ("token", "sorted"):
        out.zero_()
        moe.grouped_matmul(el, x, plan, T, top_k=1, rows=rows, out=out)
        torch.cuda.synchronize()
        for e in range(2):
            if rows == "token":
                mine = torch.nonzero(idx[:, 0] == e)[:, 0]
            else:
                c = int((idx == 0).sum())
                mine = torch.arange(c, device="cuda") if e == 0 else torch.arange(c, T, device="cuda")
            ref.check(out[mine], *ref.product(x[mine], el.w[e], out_dtype=BF16), f"{rows} e={e}")


def test_matmul_of_no_rows():
    lin = make_linear(gen(1), None, 8, 8, BF16, False, False, "none", BF16)
    assert moe.matmul(lin, torch.empty((0, 8), dtype=BF16, device="cuda")).shape == (0, 8)


# ----------------------------------------------------------------- grouped
def plan_of(idx, E):
    t = torch.as_tensor(np.asarray(idx, np.int32)).cuda()
    return t, moe.expert_plan(t, E)


def routing(rng, T, E, k, skew=0.0):
    lg = rng.standard_normal((T, E)) - skew * np.log(rng.permutation(E) + 1)
    return np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)


def check_grouped(idx, E, K, N, dtype, gated, bias, act, out_dtype, rows, clamp=0.0, x_pad=0, w_pad=0, o_pad=0, tag="",
                  seed=3):
    g = gen(seed)
    T, k = idx.shape
    n = T * k
    lin = make_linear(g, E, N, K, dtype, gated, bias, act, out_dtype, clamp, w_pad)
    flat = idx.reshape(-1)
    for e in range(E):
        if not (flat == e).any():  # nobody reads an expert without rows
            lin.w[e].fill_(float("nan"))
    _, plan = plan_of(idx, E)
    x = strided(g, T if rows == "token" else n, K, dtype, x_pad)
    out, untouched = out_view(n, N, out_dtype, o_pad)
    moe.grouped_matmul(lin, x, plan, n, top_k=k, rows=rows, out=out)
    torch.cuda.synchronize()
    order = [s for e in range(E) for s in np.nonzero(flat == e)[0]]
    want = torch.full((n, N), SENTINEL, dtype=out_dtype, device="cuda").double()
    tol = torch.zeros_like(want)
    at = 0
    for e in range(E):
        s = torch.as_tensor(np.nonzero(flat == e)[0]).cuda()
        if s.numel() == 0:
            continue
        here = torch.arange(at, at + s.numel(), device="cuda")
        at += s.numel()
        src = {"token": s // k, "slot": s, "sorted": here}[rows]
        dst = here if rows == "sorted" else s
        want[dst], tol[dst] = reference(lin, act, clamp, x[src], e=e)
    assert at == len(order)
    ref.check(out, want, tol, tag)
    untouched()


GROUPED = [  # tokens, experts, top_k, K, N, popularity skew
    (1, 4, 2, 64, 32, 0.0), (1, 128, 8, 256, 96, 0.0), (2, 8, 3, 100, 50, 0.0), (7, 3, 3, 1003, 70, 0.0),
    (8, 128, 8, 512, 128, 0.0), (32, 16, 8, 768, 256, 1.1), (33, 5, 1, 72, 33, 0.0), (64, 1, 1, 136, 65, 0.0),
    (100, 300, 6, 128, 72, 0.0), (120, 6, 2, 520, 257, 2.0), (256, 8, 2, 264, 192, 0.5), (500, 40, 4, 192, 64, 1.1),
    (700, 2, 2, 1024, 384, 0.0), (1024, 32, 8, 512, 128, 0.5), (1500, 1000, 10, 64, 24, 0.0)]


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
def test_grouped_shapes(case, rows, dtype):
    T, E, k, K, N, skew = case
    log(f"[case] grouped {case} rows={rows} {dtype}")
    idx = routing(np.random.default_rng(T + E), T, E, k, skew)
    for gated, bias, act, od in ((True, False, "silu", dtype), (False, True, "gelu", F32)):
        check_grouped(idx, E, K, N, dtype, gated, bias, act, od, rows, tag=name(case=case, rows=rows, gated=gated))


@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("T", [3, 40, 600])
def test_grouped_strides_clamp_and_fp32_rows(rows, T):
    idx = routing(np.random.default_rng(T), T, 12, 3)
    for x_pad, w_pad, o_pad in ((0, 0, 0), (8, 8, 4), (5, 0, 3), (0, 3, 0)):
        log(f"[case] grouped strides T={T} rows={rows} {x_pad},{w_pad},{o_pad}")
        check_grouped(idx, 12, 200, 72, BF16, True, True, "gelu_tanh", BF16, rows, clamp=0.8, x_pad=x_pad, w_pad=w_pad,
                      o_pad=o_pad, tag=name(T=T, rows=rows, pads=(x_pad, w_pad, o_pad)))


@pytest.mark.parametrize("T", [1, 30, 400])
def test_grouped_uneven_groups(T):
    """One expert with every row, experts with one row, first and last experts empty."""
    E, k = 9, 2
    one = np.stack([np.full(T, 4), np.where(np.arange(T) == 0, 7, 4)], axis=1).astype(np.int32)
    check_grouped(one, E, 160, 80, BF16, False, False, "none", F32, "slot", tag=f"one expert T={T}")
    check_grouped(np.full((T, k), 8, np.int32), E, 160, 80, BF16, True, False, "silu", BF16, "token", tag="the last")
    check_grouped(np.zeros((T, k), np.int32), E, 160, 80, F16, True, False, "silu", F16, "sorted", tag="the first")


@pytest.mark.parametrize("T", [1, 30, 400])
def test_grouped_leaves_rows_of_bad_experts(T):
    """Slots with an expert id outside the layer are in no group: their rows stay."""
    rng = np.random.default_rng(T)
    E, k = 10, 3
    idx = routing(rng, T, E, k)
    idx[rng.random(idx.shape) < 0.3] = E
    idx[0, 0], idx[-1, -1] = -1, 1 << 30
    check_grouped(idx, E, 96, 48, BF16, True, False, "silu", BF16, "token", tag=f"bad ids T={T}")
    check_grouped(np.full((T, k), -5, np.int32), E, 96, 48, BF16, True, False, "silu", BF16, "token", tag="all bad")


def test_grouped_ignores_a_malformed_plan():
    """Records and slots outside the plan's range are skipped: no access outside the buffers,
    which lie between sentinels."""
    g = gen(4)
    E, n, K, N = 6, 40, 64, 64
    lin = make_linear(g, E, N, K, BF16, False, False, "none", BF16)
    idx, plan = plan_of(np.arange(n, dtype=np.int32).reshape(n, 1) % E, E)
    for breakage in ("expert", "first", "count", "negative", "slots"):
        plan = moe.expert_plan(idx, E)
        if breakage == "expert":
            plan.work[2, 0] = E
        elif breakage == "first":
            plan.work[2, 1] = 1 << 30
        elif breakage == "count":
            plan.work[2, 2] = n
        elif breakage == "negative":
            plan.work[2, 1], plan.work[3, 2] = -3, -1
        else:
            plan.sorted_slots[::3] = 1 << 20
            plan.sorted_slots[1::3] = -7
        for rows in ("token", "slot"):
            x = normal(g, (n, K), BF16)
            out, untouched = out_view(n, N, BF16, 0)
            moe.grouped_matmul(lin, x, plan, n, top_k=1, rows=rows, out=out)
            torch.cuda.synchronize()
            untouched()
            full, tol = torch.empty((n, N), dtype=torch.float64, device="cuda"), torch.empty((n, N), dtype=torch.float64, device="cuda")
            for e in range(E):
                full[e::E], tol[e::E] = reference(lin, "none", 0.0, x[e::E], e=e)
            stays = (out == torch.tensor(SENTINEL, dtype=BF16, device="cuda")).all(dim=1)
            ref.check(out[~stays], full[~stays], tol[~stays], breakage)
            assert bool(stays.any()), breakage


@pytest.mark.parametrize("K", [64, 8192])
def test_grouped_keeps_to_its_workspace_when_records_overlap(K):
    """A plan whose records all claim every slot needs more tiles than any real plan of that
    many slots: what does not fit is dropped, nothing outside out and the workspace is written."""
    g = gen(4)
    E, n, N = 8, 70, 64
    lin = make_linear(g, E, N, K, BF16, False, False, "none", BF16)
    plan = moe.expert_plan(torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1) % E, E)
    plan.work[:, 1], plan.work[:, 2] = 0, n
    x = normal(g, (n, K), BF16)
    need = max(moe.grouped_workspace_size(lin, n), 256)
    buf = torch.full((need // 4 + 128,), SENTINEL, device="cuda")
    out, untouched = out_view(n, N, BF16, 0)
    moe.grouped_matmul(lin, x, plan, n, rows="slot", out=out, workspace=buf[64:-64])
    torch.cuda.synchronize()
    untouched()
    assert bool((buf[:64] == SENTINEL).all()) and bool((buf[-64:] == SENTINEL).all())


def test_grouped_same_rows_as_one_matmul():
    """An expert's rows against moe_matmul of its matrix on the same rows."""
    g = gen(21)
    E, T, K, N = 3, 90, 256, 128
    lin = make_linear(g, E, N, K, BF16, True, True, "silu", BF16)
    idx, plan = plan_of(np.arange(T, dtype=np.int32).reshape(T, 1) % E, E)
    x = normal(g, (T, K), BF16)
    out = moe.grouped_matmul(lin, x, plan, T, rows="token")
    for e in range(E):
        one = moe.Linear.from_tensors(lin.w[e], bias=lin.bias[e], w_up=lin.w_up[e], bias_up=lin.bias_up[e],
                                      activation="silu")
        ref.check(out[e::E], *ref.product(x[e::E], lin.w[e], lin.bias[e], lin.w_up[e], lin.bias_up[e], "silu",
                                          out_dtype=BF16), f"grouped e={e}")
        ref.check(moe.matmul(one, x[e::E]), *ref.product(x[e::E], lin.w[e], lin.bias[e], lin.w_up[e], lin.bias_up[e],
                                                         "silu", out_dtype=BF16), f"matmul e={e}")


def test_grouped_of_no_slots():
    lin = make_linear(gen(1), 4, 8, 8, BF16, False, False, "none", BF16)
    plan = moe.expert_plan(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4)
    assert moe.grouped_matmul(lin, torch.empty((0, 8), dtype=BF16, device="cuda"), plan, 0, top_k=2).shape == (0, 8)


# ----------------------------------------------------------------- combine
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 2048), (2, 6, 4096), (3, 16, 30), (5, 4, 101), (32, 8, 2048),
                                   (100, 5, 12), (1000, 2, 515), (4096, 3, 64)])
@pytest.mark.parametrize("y_dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
def test_combine(T, k, H, y_dtype):
    E = 20
    g = gen(T + H)
    idx = torch.as_tensor(routing(np.random.default_rng(T), T, E, k)).cuda()
    w = torch.softmax(normal(g, (T, k), F32), dim=1)
    y = normal(g, (T * k, H), y_dtype)
    for out_dtype, res_dtype in ((BF16, BF16), (F32, None), (F16, F32), (F32, F16), (BF16, None)):
        log(f"[case] combine T={T} k={k} H={H} y={y_dtype} out={out_dtype} res={res_dtype}")
        res = None if res_dtype is None else normal(g, (T, H), res_dtype)
        out, untouched = out_view(T, H, out_dtype, 0)
        moe.combine(y, idx, w, E, residual=res, out=out)
        torch.cuda.synchronize()
        ref.check(out, *ref.combine(y, idx, w, E, res, out_dtype), f"T={T} k={k} H={H}")
        untouched()


@pytest.mark.parametrize("offset", [1, 2, 3, 4])
def test_combine_at_odd_addresses_and_in_place(offset):
    g = gen(2)
    T, k, H, E = 7, 3, 64, 5
    idx = torch.as_tensor(routing(np.random.default_rng(1), T, E, k)).cuda()
    w = torch.softmax(normal(g, (T, k), F32), dim=1)
    y = strided(g, T * k, H, BF16, 0, offset=offset)
    out, untouched = out_view(T, H, BF16, 0, offset=offset)
    r = normal(g, (T, H), BF16)
    out.copy_(r)
    moe.combine(y, idx, w, E, residual=out, out=out)
    torch.cuda.synchronize()
    ref.check(out, *ref.combine(y, idx, w, E, r, BF16), f"offset {offset}")
    untouched()


def test_combine_bad_expert_ids_give_nan_rows():
    g = gen(3)
    T, k, H, E = 9, 4, 70, 6
    idx = torch.as_tensor(routing(np.random.default_rng(1), T, E, k)).cuda()
    idx[2, 1], idx[5, 3], idx[8, 0] = -1, E, 1 << 30
    w = torch.softmax(normal(g, (T, k), F32), dim=1)
    y = normal(g, (T * k, H), F32)
    y[2 * k + 1] = float("nan")
    out = moe.combine(y, idx, w, E, out_dtype=BF16)
    torch.cuda.synchronize()
    ref.check(out, *ref.combine(torch.nan_to_num(y), idx, w, E, None, BF16), "bad ids")


# ---------------------------------------------------- as they are used
def expert_block(x, logits, k, gate_up, down, shared_gu, shared_down, E, buffers=None):
    """An unquantised layer step: routed experts, a shared expert, residual."""
    b = buffers or {}
    idx, w, plan = moe.route_plan(logits, k, plan=b.get("plan"), idx=b.get("idx"), w=b.get("w"))
    n = idx.numel()
    s = moe.matmul(shared_gu, x, out=b.get("s"))
    r = moe.matmul(shared_down, s, residual=x, out=b.get("r"))
    h = moe.grouped_matmul(gate_up, x, plan, n, top_k=k, rows="token", out=b.get("h"))
    y = moe.grouped_matmul(down, h, plan, n, top_k=k, rows="slot", out=b.get("y"))
    return moe.combine(y, idx, w, E, residual=r, out=b.get("out"), out_dtype=None if b.get("out") is not None else x.dtype)


def block_weights(g, E, H, F):
    gu = make_linear(g, E, F, H, BF16, True, False, "silu", BF16)
    dn = make_linear(g, E, H, F, BF16, False, False, "none", F32)
    sgu = make_linear(g, None, F, H, BF16, True, False, "silu", BF16)
    sdn = make_linear(g, None, H, F, BF16, False, False, "none", F32)
    return gu, dn, sgu, sdn


def block_reference(x, logits, k, gu, dn, sgu, sdn):
    """The chain in 64 bits on the intermediates' stored types (h rounded to bf16 as the
    linear's out_dtype says), routing from the logits; a bound by the roundings of h
    and of out: h is off by half a step (2^-8) of each value, carried through |W_down|."""
    idx = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    w = torch.softmax(torch.gather(logits.double(), 1, idx), dim=1)

    def mlp(xs, a, b, e=None):
        wg, wu, wd = (a.w, a.w_up, b.w) if e is None else (a.w[e], a.w_up[e], b.w[e])
        g64 = xs.double() @ wg.double().t()
        h = g64 * torch.sigmoid(g64) * (xs.double() @ wu.double().t())
        return h @ wd.double().t(), 2.0 ** -8 * 1.01 * (h.abs() @ wd.double().abs().t())

    out, tol = mlp(x, sgu, sdn)
    out = out + x.double()
    for t in range(x.shape[0]):
        for j in range(k):
            v, e = mlp(x[t:t + 1], gu, dn, int(idx[t, j]))
            out[t] += w[t, j] * v[0]
            tol[t] += w[t, j] * e[0] + 1e-6 * v[0].abs()
    return out, tol + 1e-5 + ref.half_step(BF16, out.abs() + tol)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_expert_block_of_unquantised_layers(T):
    g = gen(31)
    E, k, H, F = 16, 4, 256, 192
    weights = block_weights(g, E, H, F)
    x, logits = normal(g, (T, H), BF16), normal(g, (T, E), F32)
    out = expert_block(x, logits, k, *weights, E)
    torch.cuda.synchronize()
    ref.check(out, *block_reference(x, logits, k, *weights), f"T={T}")


@pytest.mark.parametrize("T", [1, 40])
def test_expert_block_in_a_graph(T):
    """Captured once, replayed on new inputs with eager calls between: every replay is the
    eager result bit for bit; two graphs of the same layer do not disturb each other."""
    g = gen(32)
    E, k, H, F = 16, 4, 256, 192
    weights = block_weights(g, E, H, F)
    n = T * k

    def buffers():
        e = dict(device="cuda")
        return dict(plan=moe.Plan.allocate(E, n), idx=torch.empty((T, k), dtype=torch.int32, **e),
                    w=torch.empty((T, k), dtype=F32, **e), s=torch.empty((T, F), dtype=BF16, **e),
                    r=torch.empty((T, H), dtype=F32, **e), h=torch.empty((n, F), dtype=BF16, **e),
                    y=torch.empty((n, H), dtype=F32, **e), out=torch.empty((T, H), dtype=BF16, **e))

    graphs = []
    for _ in range(2):
        x, lg, b = normal(g, (T, H), BF16), normal(g, (T, E), F32), buffers()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            expert_block(x, lg, k, *weights, E, buffers=b)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            expert_block(x, lg, k, *weights, E, buffers=b)
        graphs.append((graph, x, lg, b))
    for i in range(4):
        for graph, x, lg, b in graphs:
            x.copy_(normal(g, (T, H), BF16))
            lg.copy_(normal(g, (T, E), F32))
            eager = expert_block(x, lg, k, *weights, E)
            b["out"].fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(b["out"].view(torch.int16), eager.view(torch.int16)), f"replay {i}"


def test_products_on_other_streams():
    """On a stream of the caller's, named or current, with what the call allocates."""
    g = gen(33)
    lin = make_linear(g, None, 512, 2048, BF16, True, False, "silu", BF16)
    x = normal(g, (180, 2048), BF16)
    want = moe.matmul(lin, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for i in range(6):
        outs.append(moe.matmul(lin, x, stream=s))
        with torch.cuda.stream(s):
            outs.append(moe.matmul(lin, x))
        outs.append(moe.matmul(lin, x))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


def test_wrappers_refuse_what_does_not_fit():
    g = gen(34)
    lin = make_linear(g, None, 16, 32, BF16, False, False, "none", BF16)
    x = normal(g, (4, 32), BF16)
    for bad in (normal(g, (4, 33), BF16), normal(g, (4, 32), F16), normal(g, (4, 32), BF16).cpu(),
                normal(g, (32, 4), BF16).t(), normal(g, (1, 32), BF16).expand(4, 32)):
        with pytest.raises(ValueError):
            moe.matmul(lin, bad)
    for out in (torch.empty((4, 15), dtype=BF16, device="cuda"), torch.empty((4, 16), dtype=F32, device="cuda"),
                torch.empty((1, 16), dtype=BF16, device="cuda").expand(4, 16)):
        with pytest.raises(ValueError):
            moe.matmul(lin, x, out=out)
    with pytest.raises(ValueError):
        moe.matmul(lin, x, residual=normal(g, (4, 15), BF16))
    with pytest.raises(moe.MoeError):  # out over x
        moe.matmul(lin, x, out=x[:, :16])
    el = make_linear(g, 4, 16, 32, BF16, False, False, "none", BF16)
    with pytest.raises(moe.MoeError):
        moe.matmul(el, x)
    idx, plan = plan_of(np.zeros((4, 2), np.int32), 4)
    with pytest.raises(ValueError):
        moe.grouped_matmul(el, x, plan, 9, top_k=2)
    with pytest.raises(ValueError):
        moe.grouped_matmul(el, x, plan, 8, top_k=2, rows="slot")
    with pytest.raises(ValueError):
        moe.grouped_matmul(el, x, plan, 8, top_k=2, rows="columns")
    _, short = plan_of(np.zeros((4, 1), np.int32), 4)
    with pytest.raises(ValueError):
        moe.grouped_matmul(el, x, short, 8, top_k=2)
    w = torch.ones((4, 2), device="cuda")
    for y in (normal(g, (7, 16), F32), normal(g, (8, 16), F32).cpu(), normal(g, (16, 8), F32).t()):
        with pytest.raises(ValueError):
            moe.combine(y, idx, w, 4)


def test_wrappers_refuse_sizes_past_32_bits():
    n = 2 ** 32 + 5  # 5 in the ABI's 32 bits
    x = torch.empty((n, 1), dtype=BF16, device="cuda")
    g = gen(35)
    lin = make_linear(g, None, 8, 1, BF16, False, False, "none", BF16)
    with pytest.raises(ValueError):
        moe.matmul(lin, x, out=torch.empty((5, 8), dtype=BF16, device="cuda"))
    for w in (x, x.view(1, n, 1), x.view(n, 1, 1)):
        with pytest.raises(ValueError):
            moe.Linear.from_tensors(w)
    del x
    el = make_linear(g, 4, 16, 32, BF16, False, False, "none", BF16)
    idx, plan = plan_of(np.zeros((4, 2), np.int32), 4)
    with pytest.raises(ValueError):
        moe.grouped_matmul(el, normal(g, (4, 32), BF16), plan, 8, top_k=2 ** 32 + 2)
    with pytest.raises(ValueError):
        moe.combine(normal(g, (8, 16), F32), idx, torch.ones((4, 2), device="cuda"), 2 ** 32 + 4)
