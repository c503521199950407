"""moe_quantize_rows, moe_matmul_int and moe_grouped_matmul_int on the GPU against their definitions
in 64 bits (int_ref.py derives the tolerances)."""

import numpy as np
import pytest
import torch

import int_ref as ref
import quantized_expert_gemv_moe_amd as moe
from gpu_helpers import log

pytestmark = pytest.mark.gpu

BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
SENTINEL = 12345.0  # compared as stored
TYPES = [BF16, F16, F32]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=F32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def codes(g, shape, lo=-128):
    return torch.randint(lo, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(I8)


def uniform(g, shape, lo, hi):
    return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g)


def strided(values, pad, offset=0, fill=None):
    """`values` [rows, cols] as a view of a wider buffer filled with NaN (integers: 99), `offset` elements in."""
    rows, cols = values.shape
    fill = (99 if values.dtype is I8 else float("nan")) if fill is None else fill
    buf = torch.full((rows * (cols + pad) + offset + 64,), fill, dtype=values.dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(values)
    return v


def out_view(rows, cols, dtype, pad=0, offset=0):
    """An out view inside a sentinel-filled buffer, and a check that only the view was written."""
    fill = 55 if dtype is I8 else SENTINEL
    buf = torch.full((rows * (cols + pad) + offset + 64,), fill, dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    def untouched():
        mine = torch.zeros_like(buf, dtype=torch.bool)
        mine[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = True
        s = torch.tensor(fill, dtype=dtype, device="cuda")
        assert bool((buf[~mine] == s).all()), "wrote outside out"

    return v, untouched


def make_linear(g, E, N, K, gated=False, bias=None, act="none", out_dtype=BF16, clamp=0.0, w_pad=0):
    lead = () if E is None else (E,)

    def mat():
        m = torch.full(lead + (N, K + w_pad), 99, dtype=I8, device="cuda")[..., :K]
        m.copy_(codes(g, lead + (N, K)))
        return m

    def vec():
        return uniform(g, lead + (N,), 0.5 / 74 / K ** 0.5, 1.5 / 74 / K ** 0.5)  # uniform codes: std 74

    w, ws = mat(), vec()
    up, ups = (mat(), vec()) if gated else (None, None)
    b = None if bias is None else normal(g, lead + (N,), bias, 0.5)
    bu = normal(g, lead + (N,), bias, 0.5) if bias is not None and gated else None
    return moe.LinearInt.from_tensors(w, ws, bias=b, w_up=up, w_up_scale=ups, bias_up=bu, activation=act,
                                      out_dtype=out_dtype, clamp_limit=clamp)


def make_x(g, rows, K, dtype):
    """(x, x_scale or None, codes in fp64, scales)."""
    if dtype is I8:
        x, s = codes(g, (rows, K)), uniform(g, (rows,), 0.01, 0.03)
        return x, s, x.double(), s
    x = normal(g, (rows, K), dtype)
    q, s = ref.quantize(x)
    return x, None, q, s


def reference(lin, act, clamp, q, s, residual=None, e=None):
    def pick(t):
        return t if t is None or e is None else t[e]

    return ref.product(q, s, pick(lin.w), pick(lin.w_scale), pick(lin.bias), pick(lin.w_up), pick(lin.w_up_scale),
                       pick(lin.bias_up), act, clamp, residual, lin.out_dtype)


def name(**kw):
    return " ".join(f"{k}={v}" for k, v in kw.items())


# ---------------------------------------------------------------- quantise
def check_quantize(x, tag, **kw):
    q, s = moe.quantize_rows(x, **kw)
    torch.cuda.synchronize()
    want_q, want_s = ref.quantize(x)
    assert q.dtype is I8 and s.dtype is F32
    bad = q.double() != want_q
    assert not bool(bad.any()), f"{tag}: {int(bad.sum())} codes differ, first {q[bad][0]} for {want_q[bad][0]}"
    assert torch.equal(s.view(torch.int32) & 0x7FFFFFFF, want_s.view(torch.int32) & 0x7FFFFFFF) or (
        torch.equal(torch.isnan(s), torch.isnan(want_s)) and torch.equal(s[~torch.isnan(s)], want_s[~torch.isnan(want_s)])), tag


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [1, 3, 8, 15, 64, 100, 512, 520, 1003, 1024, 1032, 2048, 4099, 8192, 16384, 20011, 70000])
def test_quantize_rows(cols, dtype):
    log(f"[case] quantize cols={cols} {dtype}")
    for rows in (1, 4, 5, 130):
        g = gen(cols + rows)
        check_quantize(normal(g, (rows, cols), dtype), name(rows=rows, cols=cols))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
def test_quantize_halves_go_to_even(dtype):
    """Quotients half way between two integers, and just beside it."""
    log(f"[case] quantize halves {dtype}")
    k = torch.arange(-127, 127, device="cuda", dtype=F32) + 0.5
    rows = []
    for p in (-20, -3, 0, 5):
        if dtype is F16 and p == -20:
            p = -8
        for m in (127.0, 63.5, 254.0):
            r = torch.cat([k * (m / 127.0), torch.tensor([m], device="cuda")]) * 2.0 ** p
            rows.append(r)
            if dtype is F32:
                rows += [torch.nextafter(r, torch.full_like(r, 9e9)).clamp(-m * 2.0 ** p, m * 2.0 ** p),
                         torch.nextafter(r, torch.full_like(r, -9e9)).clamp(-m * 2.0 ** p, m * 2.0 ** p)]
    # every 8-bit mantissa against every other: all ties that bf16 can have
    a = torch.arange(128, 256, device="cuda", dtype=F32)
    for d in range(8):
        rows += list(torch.cat([a[None, :].expand(128, 128) * 2.0 ** -d, a[:, None] * 2.0], dim=1))
    width = max(r.numel() for r in rows)
    x = torch.stack([torch.cat([r, torch.zeros(width - r.numel(), device="cuda")]) for r in rows]).to(dtype)
    check_quantize(x, "halves")


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
def test_quantize_extremes(dtype):
    """Rows of zeros, of the smallest and largest numbers, with infinities and NaN anywhere."""
    log(f"[case] quantize extremes {dtype}")
    fi = torch.finfo(dtype)
    g = gen(7)
    for cols in (40, 1000, 9000):
        x = normal(g, (16, cols), dtype)
        x[1] = 0
        x[2] = -0.0
        x[3, cols - 1] = float("inf")
        x[4, 0] = float("-inf")
        x[5, cols // 2] = float("nan")
        x[6] = fi.smallest_normal
        x[7] = torch.where(torch.arange(cols, device="cuda") % 2 == 0, fi.max, fi.min).to(dtype)
        x[8] = 0
        x[8, 3] = fi.tiny * fi.eps  # the smallest subnormal
        x[9] = (normal(g, (cols,), F32) * fi.tiny).to(dtype)
        x[10] = (normal(g, (cols,), F32).clamp(-2, 2) * (fi.max / 2)).to(dtype)
        x[11, 5] = fi.max
        x[12] = fi.tiny * fi.eps * 3
        x[13, 1:] = 0
        check_quantize(x, name(cols=cols))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
def test_quantize_strides_and_given_outputs(dtype):
    log(f"[case] quantize strides {dtype}")
    for rows, cols, pad, offset, q_pad, q_off in ((3, 64, 0, 1, 0, 1), (9, 1003, 5, 3, 3, 2), (70, 2048, 8, 8, 16, 16),
                                                  (5, 4100, 1, 0, 0, 5), (2, 7, 2, 1, 1, 1)):
        g = gen(rows)
        x = strided(normal(g, (rows, cols), dtype), pad, offset)
        q, untouched = out_view(rows, cols, I8, q_pad, q_off)
        buf = torch.full((rows + 16,), SENTINEL, device="cuda")
        got = moe.quantize_rows(x, codes=q, scales=buf[8:8 + rows])
        assert got[0] is q
        check_quantize(x, name(cols=cols, pad=pad), codes=q, scales=buf[8:8 + rows])
        untouched()
        assert bool((buf[:8] == SENTINEL).all()) and bool((buf[8 + rows:] == SENTINEL).all())


def test_quantize_many_rows_and_none():
    log("[case] quantize many rows")
    check_quantize(normal(gen(1), (300001, 24), BF16), "300001 rows")
    q, s = moe.quantize_rows(torch.empty((0, 8), device="cuda"))
    assert q.shape == (0, 8) and s.shape == (0,)


def test_quantize_rows_past_4_gib():
    log("[case] quantize far rows")
    big = torch.empty((1100, 1 << 22), dtype=BF16, device="cuda")[:, :48]
    big.copy_(normal(gen(2), (1100, 48), BF16))
    check_quantize(big, "far rows")


# ------------------------------------------------------------------ matmul
SHAPES = [(1, 1, 1), (1, 16, 16), (1, 2048, 768), (2, 64, 64), (3, 7, 5), (5, 100, 33), (16, 768, 2048), (17, 80, 130),
          (31, 1003, 257), (33, 40, 48), (64, 64, 64), (65, 528, 65), (77, 1003, 1357), (128, 144, 96),
          (129, 2048, 129), (200, 8208, 72), (256, 256, 256), (300, 256, 500), (513, 333, 127), (700, 1024, 640),
          (1024, 2048, 768)]


@pytest.mark.parametrize("x_dtype", [BF16, F16, F32, I8], ids=["bf16", "fp16", "fp32", "int8"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matmul_int_shapes(shape, gated, x_dtype):
    rows, K, N = shape
    log(f"[case] matmul_int {shape} gated={gated} {x_dtype}")
    g = gen(rows * 7 + K + N)
    lin = make_linear(g, None, N, K, gated, BF16, "silu", BF16)
    x, xs, q, s = make_x(g, rows, K, x_dtype)
    res = normal(g, (rows, N), BF16)
    out, untouched = out_view(rows, N, BF16)
    got = moe.matmul_int(lin, x, x_scale=xs, residual=res, out=out)
    torch.cuda.synchronize()
    assert got is out
    ref.check(out, *reference(lin, "silu", 0.0, q, s, res), name(shape=shape, gated=gated, x=x_dtype))
    untouched()


# ends inside row and column tiles and steps, odd and even counts of whole steps, for the large tiles
LARGE = [(4090, 1152, 4000, False, BF16), (8000, 2064, 2000, False, F16), (4090, 640, 2000, True, BF16),
         (8000, 528, 1000, True, F16), (4096, 1152, 4096, False, F32), (4100, 1152, 4104, False, BF16),
         (4100, 1168, 2056, True, F16), (2001, 1003, 2000, False, BF16), (4096, 1024, 2048, True, F32)]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: "x".join(map(str, c[:4])))
@pytest.mark.parametrize("act,bias,residual", [("none", None, False), ("silu", F32, True), ("gelu", F16, False),
                                               ("gelu_tanh", BF16, True), ("relu", None, True)])
def test_matmul_int_large(case, act, bias, residual):
    rows, K, N, gated, out_dtype = case
    log(f"[case] matmul_int large {case} {act}")
    g = gen(rows + K)
    lin = make_linear(g, None, N, K, gated, bias, act, out_dtype, clamp=0.8 if act == "gelu_tanh" else 0.0)
    x, xs, q, s = make_x(g, rows, K, I8)
    res = normal(g, (rows, N), out_dtype) if residual else None
    out, untouched = out_view(rows, N, out_dtype)
    moe.matmul_int(lin, x, x_scale=xs, residual=res, out=out)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, act, 0.8 if act == "gelu_tanh" else 0.0, q, s, res), name(case=case, act=act))
    untouched()


LONG = [(1, 32768, 64), (20, 16384, 96), (64, 16384, 512), (100, 8208, 130), (300, 32784, 64), (3, 131071, 5)]


@pytest.mark.parametrize("x_dtype", [BF16, I8], ids=["bf16", "int8"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_matmul_int_long_inputs(shape, gated, x_dtype):
    """The workspace full of garbage, exactly as large as asked for and between sentinels."""
    rows, K, N = shape
    log(f"[case] long int {shape} gated={gated} {x_dtype}")
    g = gen(rows + K + N)
    lin = make_linear(g, None, N, K, gated, F32, "silu", F32)
    x, xs, q, s = make_x(g, rows, K, x_dtype)
    res = normal(g, (rows, N), F32)
    need = moe.matmul_int_workspace_size(lin, rows)
    buf = torch.full((need // 4 + 128,), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    out, untouched = out_view(rows, N, F32)
    moe.matmul_int(lin, x, x_scale=xs, residual=res, out=out, workspace=buf[64:-64])
    again = moe.matmul_int(lin, x, x_scale=xs, residual=res)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "silu", 0.0, q, s, res), name(shape=shape, gated=gated, x=x_dtype))
    assert torch.equal(out, again)
    assert bool((buf[:64] == 0x5A5A5A5A).all()) and bool((buf[-64:] == 0x5A5A5A5A).all()), "wrote outside the workspace"
    untouched()


def test_largest_sums_are_exact():
    """-128 times -128 over as many inputs as are allowed: 2^31 - 16384."""
    log("[case] largest sums")
    K = 131071
    for rows, N in ((1, 3), (40, 33), (300, 200)):
        w = torch.full((N, K), -128, dtype=I8, device="cuda")
        x = torch.full((rows, K), -128, dtype=I8, device="cuda")
        x[0, :], w[0, :] = 127, -128
        lin = moe.LinearInt.from_tensors(w, torch.ones(N, device="cuda"), out_dtype=F32)
        out = moe.matmul_int(lin, x, x_scale=torch.ones(rows, device="cuda"))
        torch.cuda.synchronize()
        want = (x.double() @ w.double().t()).float()  # one rounding
        assert torch.equal(out, want)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("out_dtype", TYPES, ids=["obf16", "ofp16", "ofp32"])
@pytest.mark.parametrize("rows", [3, 70])
def test_matmul_int_functions_and_output_types(rows, out_dtype, act):
    log(f"[case] matmul_int act={act} out={out_dtype} rows={rows}")
    g = gen(11)
    for gated, clamp, res_dtype, bias in ((False, 0.0, None, None), (True, 0.0, F32, BF16), (True, 0.75, BF16, F32),
                                          (False, 1.5, F16, F16)):
        lin = make_linear(g, None, 88, 192, gated, bias, act, out_dtype, clamp)
        x, xs, q, s = make_x(g, rows, 192, BF16)
        res = None if res_dtype is None else normal(g, (rows, 88), res_dtype)
        out = moe.matmul_int(lin, x, residual=res)
        torch.cuda.synchronize()
        assert out.dtype == out_dtype
        ref.check(out, *reference(lin, act, clamp, q, s, res), name(act=act, gated=gated, clamp=clamp))


@pytest.mark.parametrize("rows,K,N", [(1, 256, 48), (9, 131, 100), (40, 272, 72), (150, 1003, 200), (300, 1024, 384)])
@pytest.mark.parametrize("x_dtype", [BF16, F32, I8], ids=["bf16", "fp32", "int8"])
def test_matmul_int_strides_and_offsets(rows, K, N, x_dtype):
    """Rows of x, w, residual and out apart and at every offset; nothing outside the rows counts."""
    for x_pad, w_pad, o_pad, offset in ((0, 0, 0, 1), (16, 16, 4, 0), (3, 0, 1, 3), (0, 5, 2, 0), (64, 64, 64, 16)):
        log(f"[case] int strides rows={rows} K={K} N={N} {x_dtype} pads={x_pad},{w_pad},{o_pad} offset={offset}")
        g = gen(rows + x_pad)
        lin = make_linear(g, None, N, K, True, BF16, "gelu_tanh", BF16, w_pad=w_pad)
        x0, xs, q, s = make_x(g, rows, K, x_dtype)
        x = strided(x0, x_pad, offset)
        res = strided(normal(g, (rows, N), F16), o_pad, offset)
        out, untouched = out_view(rows, N, BF16, o_pad, offset)
        moe.matmul_int(lin, x, x_scale=xs, residual=res, out=out)
        torch.cuda.synchronize()
        ref.check(out, *reference(lin, "gelu_tanh", 0.0, q, s, res), name(pads=(x_pad, w_pad, o_pad, offset)))
        untouched()


def test_rows_without_numbers_stay_their_own():
    """A row of x with an infinity or NaN is NaN throughout, a row of zeros is f(bias), and the others do
    not notice."""
    log("[case] int rows without numbers")
    for rows, K, N in ((6, 256, 64), (200, 2048, 512)):
        g = gen(rows)
        lin = make_linear(g, None, N, K, False, BF16, "silu", F32)
        x, _, _, _ = make_x(g, rows, K, BF16)
        clean = moe.matmul_int(lin, x)
        x[1, 5], x[2, K - 1], x[4] = float("nan"), float("inf"), 0
        out = moe.matmul_int(lin, x)
        torch.cuda.synchronize()
        q, s = ref.quantize(x)
        ref.check(out, *reference(lin, "silu", 0.0, q, s), name(rows=rows))
        assert bool(torch.isnan(out[[1, 2]]).all()) and bool(torch.isfinite(out[4]).all())
        rest = [r for r in range(rows) if r not in (1, 2, 4)]
        assert torch.equal(out[rest], clean[rest])


def test_halves_of_one_buffer_and_in_place_residual():
    log("[case] int halves of one buffer")
    for rows in (2, 100, 600):
        g = gen(rows)
        K, N = 512, 256
        stack, scales = codes(g, (2 * N, K)), uniform(g, (2 * N,), 1e-4, 3e-4)
        lin = moe.LinearInt.from_tensors(stack[:N], scales[:N], w_up=stack[N:], w_up_scale=scales[N:], activation="silu")
        both = torch.empty((rows, K + N), dtype=BF16, device="cuda")
        x, out = both[:, :K], both[:, K:]
        x.copy_(normal(g, (rows, K), BF16))
        q, s = ref.quantize(x)
        moe.matmul_int(lin, x, out=out)
        torch.cuda.synchronize()
        ref.check(out, *reference(lin, "silu", 0.0, q, s), f"halves {rows}")
        res = normal(g, (rows, N), BF16)
        kept = res.clone()
        moe.matmul_int(lin, x, residual=res, out=res)
        torch.cuda.synchronize()
        ref.check(res, *reference(lin, "silu", 0.0, q, s, kept), f"in place {rows}")


def test_matmul_int_of_no_rows():
    lin = make_linear(gen(1), None, 16, 32)
    out = moe.matmul_int(lin, torch.empty((0, 32), dtype=BF16, device="cuda"))
    assert out.shape == (0, 16)


def test_quantised_beforehand_is_the_same():
    """x as it is and its own codes and scales: bit for bit the same, where the same kernel runs."""
    log("[case] int quantised beforehand")
    for rows in (1, 50, 700):
        g = gen(rows)
        lin = make_linear(g, None, 640, 1024, True, BF16, "silu", BF16)
        x = normal(g, (rows, 1024), F16)
        q, s = moe.quantize_rows(x)
        a, b = moe.matmul_int(lin, x), moe.matmul_int(lin, q, x_scale=s)
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ----------------------------------------------------------------- grouped
def plan_of(idx, E):
    t = torch.from_numpy(idx).cuda()
    return t, moe.expert_plan(t, E)


def routing(rng, T, E, k, skew=0.0):
    lg = rng.standard_normal((T, E)) - skew * np.log(rng.permutation(E) + 1)
    return np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)


def check_grouped(idx, E, K, N, x_dtype, gated, bias, act, out_dtype, rows, clamp=0.0, x_pad=0, w_pad=0, o_pad=0, tag="",
                  seed=3):
    g = gen(seed)
    T, k = idx.shape
    n = T * k
    lin = make_linear(g, E, N, K, gated, bias, act, out_dtype, clamp, w_pad)
    flat = idx.reshape(-1)
    for e in range(E):
        if not (flat == e).any():  # nobody reads an expert without rows
            lin.w_scale[e].fill_(float("nan"))
    _, plan = plan_of(idx, E)
    x0, xs, q, s = make_x(g, T if rows == "token" else n, K, x_dtype)
    x = strided(x0, x_pad)
    out, untouched = out_view(n, N, out_dtype, o_pad)
    moe.grouped_matmul_int(lin, x, plan, n, top_k=k, rows=rows, x_scale=xs, out=out)
    torch.cuda.synchronize()
    want = torch.full((n, N), SENTINEL, dtype=out_dtype, device="cuda").double()
    tol = torch.zeros_like(want)
    at = 0
    for e in range(E):
        slots = torch.as_tensor(np.nonzero(flat == e)[0]).cuda()
        if slots.numel() == 0:
            continue
        here = torch.arange(at, at + slots.numel(), device="cuda")
        at += slots.numel()
        src = {"token": slots // k, "slot": slots, "sorted": here}[rows]
        dst = here if rows == "sorted" else slots
        want[dst], tol[dst] = reference(lin, act, clamp, q[src], s[src], e=e)
    ref.check(out, want, tol, tag)
    untouched()


GROUPED = [  # tokens, experts, top_k, K, N, popularity skew
    (1, 4, 2, 64, 32, 0.0), (1, 128, 8, 256, 96, 0.0), (2, 8, 3, 100, 50, 0.0), (7, 3, 3, 1003, 70, 0.0),
    (8, 128, 8, 512, 128, 0.0), (32, 16, 8, 768, 256, 1.1), (33, 5, 1, 80, 33, 0.0), (64, 1, 1, 144, 65, 0.0),
    (100, 300, 6, 128, 72, 0.0), (120, 6, 2, 528, 257, 2.0), (256, 8, 2, 272, 192, 0.5), (500, 40, 4, 192, 64, 1.1),
    (700, 2, 2, 1024, 384, 0.0), (1024, 32, 8, 512, 128, 0.5), (1500, 1000, 10, 64, 24, 0.0)]


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("x_dtype", [BF16, F32, I8], ids=["bf16", "fp32", "int8"])
def test_grouped_int_shapes(case, rows, x_dtype):
    T, E, k, K, N, skew = case
    log(f"[case] grouped_int {case} rows={rows} {x_dtype}")
    idx = routing(np.random.default_rng(T + E), T, E, k, skew)
    for gated, act in ((True, "silu"), (False, "none")):
        check_grouped(idx, E, K, N, x_dtype, gated, BF16 if gated else None, act, BF16, rows,
                      tag=name(case=case, rows=rows, x=x_dtype, gated=gated))


# large tiles and the tile between, per expert
GROUPED_LARGE = [(3050, 3, 2, 1152, 2000, False, BF16), (3050, 3, 2, 640, 1000, True, F16), (3000, 3, 2, 1040, 1000, True, F32),
                 (2048, 16, 4, 2048, 768, True, BF16), (2000, 16, 4, 784, 2000, False, F32)]


@pytest.mark.parametrize("case", GROUPED_LARGE, ids=lambda c: "x".join(map(str, c[:6])))
@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
def test_grouped_int_large(case, rows):
    T, E, k, K, N, gated, out_dtype = case
    log(f"[case] grouped_int large {case} rows={rows}")
    idx = routing(np.random.default_rng(T), T, E, k, 0.3)
    check_grouped(idx, E, K, N, F16, gated, F32, "silu" if gated else "none", out_dtype, rows,
                  tag=name(case=case, rows=rows))


@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("T", [3, 40, 600])
def test_grouped_int_strides_and_clamp(rows, T):
    idx = routing(np.random.default_rng(T), T, 12, 3, 1.0)
    for x_dtype, x_pad, w_pad, o_pad in ((BF16, 8, 16, 4), (I8, 16, 0, 3), (I8, 3, 5, 0), (F32, 1, 32, 8)):
        log(f"[case] grouped_int strides T={T} rows={rows} {x_dtype} {x_pad},{w_pad},{o_pad}")
        check_grouped(idx, 12, 320, 100, x_dtype, True, F16, "gelu_tanh", F32, rows, clamp=1.5, x_pad=x_pad, w_pad=w_pad,
                      o_pad=o_pad, tag=name(T=T, rows=rows, x=x_dtype))


@pytest.mark.parametrize("rows", ["token", "slot", "sorted"])
@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (3, 4, 2), (40, 3, 2)])
def test_grouped_int_long_inputs(T, E, k, rows):
    idx = routing(np.random.default_rng(T), T, E, k)
    for x_dtype, gated in ((BF16, True), (I8, False)):
        log(f"[case] grouped_int long T={T} rows={rows} {x_dtype}")
        check_grouped(idx, E, 16384, 64, x_dtype, gated, BF16, "silu", BF16, rows, tag=name(T=T, rows=rows))


@pytest.mark.parametrize("T", [1, 30, 400])
def test_grouped_int_leaves_rows_of_bad_experts(T):
    log(f"[case] grouped_int bad experts T={T}")
    idx = routing(np.random.default_rng(T), T, 6, 2)
    idx[0, 1], idx[T // 2, 0] = -1, 6
    check_grouped(idx, 6, 256, 64, BF16, True, None, "silu", BF16, "token", tag=f"bad experts T={T}")


def test_grouped_int_ignores_a_malformed_plan():
    """Records and slots out of range never lead out of bounds, and rows that they do not list stay."""
    log("[case] grouped_int malformed plan")
    g = gen(9)
    E, k, T, K, N = 4, 2, 8, 128, 64
    n = T * k
    lin = make_linear(g, E, N, K)
    idx = routing(np.random.default_rng(0), T, E, k)
    _, good = plan_of(idx, E)
    x, xs, _, _ = make_x(g, T, K, I8)
    want = moe.grouped_matmul_int(lin, x, good, n, top_k=k, x_scale=xs)
    for change in ("expert", "first", "count", "slot", "slot_low"):
        _, plan = plan_of(idx, E)
        if change == "expert":
            plan.work[1, 0] = 77
        elif change == "first":
            plan.work[1, 1] = n
        elif change == "count":
            plan.work[1, 2] = 1 << 20
        else:
            plan.sorted_slots[3] = 1000 if change == "slot" else -5
        out, untouched = out_view(n, N, BF16)
        moe.grouped_matmul_int(lin, x, plan, n, top_k=k, x_scale=xs, out=out)
        torch.cuda.synchronize()
        untouched()
        same = (out == want).all(dim=1) | (out == SENTINEL).all(dim=1) | (out == torch.tensor(SENTINEL, dtype=BF16)).all(dim=1)
        assert bool(same.all()), change


def test_grouped_int_of_no_slots():
    g = gen(2)
    lin = make_linear(g, 4, 16, 32)
    plan = moe.Plan.allocate(4, 1)
    out = moe.grouped_matmul_int(lin, torch.empty((0, 32), dtype=BF16, device="cuda"), plan, 0, top_k=2)
    assert out.shape == (0, 16)


def test_x_gathered_over_4_gib():
    """Tokens whose integers alone take more than 4 GiB: rows by token through the kernel for far rows."""
    log("[case] int far rows")
    E, k, K, N, T, stride = 4, 2, 64, 32, 1100, 1 << 22
    g = gen(4)
    idx = routing(np.random.default_rng(1), T, E, k)
    _, plan = plan_of(idx, E)
    lin = make_linear(g, E, N, K)
    x = torch.empty((T, stride), dtype=I8, device="cuda")[:, :K]
    x.copy_(codes(g, (T, K)))
    s = uniform(g, (T,), 0.01, 0.02)
    out = moe.grouped_matmul_int(lin, x, plan, T * k, top_k=k, x_scale=s)
    near = moe.grouped_matmul_int(lin, x.contiguous(), plan, T * k, top_k=k, x_scale=s)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), near.view(torch.int16))


# -------------------------------------------------------- together, as used
def block(x, logits, router, gu, dn, sgu, sdn, buffers=None):
    """A routed layer of 8-bit experts beside a shared one: router and plan, gated gate+up, down into fp32
    rows, shared expert as the residual, combine."""
    b = buffers or {}
    idx, w, plan = moe.router_plan(router, logits, plan=b.get("plan"), idx=b.get("idx"), w=b.get("w"))
    n, k = idx.numel(), idx.shape[1]
    s = moe.matmul_int(sgu, x, out=b.get("s"), workspace=b.get("ws1"))
    r = moe.matmul_int(sdn, s, residual=x, out=b.get("r"), workspace=b.get("ws2"))
    h = moe.grouped_matmul_int(gu, x, plan, n, top_k=k, rows="token", out=b.get("h"), workspace=b.get("ws3"))
    y = moe.grouped_matmul_int(dn, h, plan, n, rows="slot", out=b.get("y"), workspace=b.get("ws4"))
    return moe.combine(y, idx, w, router.n_experts, residual=r, out=b.get("out"), out_dtype=BF16), idx, w


def layer(g, E, H, F):
    return (make_linear(g, E, F, H, True, None, "silu", BF16), make_linear(g, E, H, F, out_dtype=F32),
            make_linear(g, None, F, H, True, None, "silu", BF16), make_linear(g, None, H, F, out_dtype=F32))


def layer_reference(x, logits, router, gu, dn, sgu, sdn):
    """The block with every rounding point where the calls have it (h and s rounded to bf16 and quantised
    again), from 64-bit values; and a tolerance for its sum."""
    import router_ref

    bias = None if router.bias is None else router.bias.double().cpu().numpy()
    ids, w, _ = router_ref.route(logits.double().cpu().numpy(), "fp32", router.top_k, router.score, bias, router.n_groups,
                                 router.top_groups, router.group_score, router.renormalise, router.scale)
    q, s = ref.quantize(x)
    hs = reference(sgu, "silu", 0.0, q, s)[0].to(BF16)
    out = reference(sdn, "none", 0.0, *ref.quantize(hs))[0] + x.double()
    for t in range(x.shape[0]):
        for j in range(router.top_k):
            e = int(ids[t, j])
            h = reference(gu, "silu", 0.0, q[t:t + 1], s[t:t + 1], e=e)[0].to(BF16)
            out[t] += w[t, j] * reference(dn, "none", 0.0, *ref.quantize(h), e=e)[0][0]
    return out, ids


@pytest.mark.parametrize("T", [1, 5, 40])
def test_expert_block_of_integer_layers(T):
    """Against 64 bits.  A value of h next to a rounding point of bf16 may fall on the other side, half a step
    (2^-8) of it, and a code of it by one (1 / 127 of the row's largest): both sides of such a point are right,
    and the block's norm moves by far less than the 2e-3 that the 4-bit block is held to."""
    log(f"[case] int block T={T}")
    g = gen(T)
    E, H, F, k = 24, 256, 192, 6
    weights = layer(g, E, H, F)
    x, logits = normal(g, (T, H), BF16), normal(g, (T, E), F32)
    bias = normal(g, (E,), F32, 0.1)
    router = moe.Router(E, k, score="sigmoid", bias=bias, n_groups=4, top_groups=2, group_score="top2", scale=2.0)
    out, idx, _ = block(x, logits, router, *weights)
    torch.cuda.synchronize()
    want, ids = layer_reference(x, logits, router, *weights)
    assert np.array_equal(idx.cpu().numpy(), ids)
    err = float((out.double() - want).norm() / want.norm())
    assert err <= 2.0 ** -9 + 2e-3, err  # the output's own rounding and the block's


@pytest.mark.parametrize("T", [1, 40])
def test_expert_block_in_a_graph(T):
    """Captured once, replayed on new inputs with eager calls between: every replay is the eager
    result bit for bit; two graphs with workspaces of their own do not disturb each other."""
    log(f"[case] int block graph T={T}")
    g = gen(32)
    E, k, H, F = 16, 4, 256, 192
    weights = layer(g, E, H, F)
    gu, dn, sgu, sdn = weights
    router = moe.Router(E, k, score="sigmoid", bias=normal(g, (E,), F32, 0.1))
    n = T * k

    def buffers():
        e = dict(device="cuda")
        return dict(plan=moe.Plan.allocate(E, n), idx=torch.empty((T, k), dtype=torch.int32, **e),
                    w=torch.empty((T, k), dtype=F32, **e), s=torch.empty((T, F), dtype=BF16, **e),
                    r=torch.empty((T, H), dtype=F32, **e), h=torch.empty((n, F), dtype=BF16, **e),
                    y=torch.empty((n, H), dtype=F32, **e), out=torch.empty((T, H), dtype=BF16, **e),
                    ws1=moe.alloc_matmul_int_workspace(sgu, T), ws2=moe.alloc_matmul_int_workspace(sdn, T),
                    ws3=moe.alloc_grouped_int_workspace(gu, n, T), ws4=moe.alloc_grouped_int_workspace(dn, n))

    graphs = []
    for _ in range(2):
        x, lg, b = normal(g, (T, H), BF16), normal(g, (T, E), F32), buffers()
        block(x, lg, router, *weights, buffers=b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block(x, lg, router, *weights, buffers=b)
        graphs.append((graph, x, lg, b))
    for i in range(4):
        for graph, x, lg, b in graphs:
            x.copy_(normal(g, (T, H), BF16))
            lg.copy_(normal(g, (T, E), F32))
            eager = block(x, lg, router, *weights)[0]
            b["out"].fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(b["out"].view(torch.int16), eager.view(torch.int16)), f"replay {i}"


def test_integer_products_on_other_streams():
    log("[case] int streams")
    g = gen(33)
    lin = make_linear(g, None, 512, 2048, True, None, "silu", BF16)
    for rows in (2, 180):
        x = normal(g, (rows, 2048), BF16)
        want = moe.matmul_int(lin, x)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        outs = []
        for _ in range(6):
            outs.append(moe.matmul_int(lin, x, stream=s))
            with torch.cuda.stream(s):
                outs.append(moe.matmul_int(lin, x))
            outs.append(moe.matmul_int(lin, x))
        q = moe.quantize_rows(x, stream=s)
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o.view(torch.int16), want.view(torch.int16))
        assert torch.equal(q[0], moe.quantize_rows(x)[0])


def test_weights_are_made_by_quantize_rows():
    """A layer from floating weights, and how near it is to them: codes are off by half a step at most, so an
    output is off by at most sum (|x| sw + |w| sx + sx sw / 2) / 2."""
    log("[case] int weights made")
    g = gen(3)
    rows, K, N = 20, 500, 96
    w, x = normal(g, (N, K), BF16, 0.05), normal(g, (rows, K), BF16)
    q, s = moe.quantize_rows(w)
    lin = moe.LinearInt.from_tensors(q, s, out_dtype=F32)
    out = moe.matmul_int(lin, x)
    torch.cuda.synchronize()
    _, sx = ref.quantize(x)
    xd, wd = x.double(), w.double()
    bound = 0.5 * (xd.abs().sum(1)[:, None] * s.double()[None, :] + sx.double()[:, None] * wd.abs().sum(1)[None, :]
                   + 0.5 * K * sx.double()[:, None] * s.double()[None, :])
    assert bool(((out.double() - xd @ wd.t()).abs() <= 1.001 * bound).all())


def test_wrappers_refuse_what_does_not_fit():
    g = gen(34)
    lin = make_linear(g, None, 16, 32)
    x = normal(g, (4, 32), BF16)
    xq, xs = moe.quantize_rows(x)
    for bad in (normal(g, (4, 33), BF16), x.double(), x.cpu(), normal(g, (32, 4), BF16).t(), x[:1].expand(4, 32), xq):
        with pytest.raises(ValueError):
            moe.matmul_int(lin, bad)
    for sc in (xs[:3], xs.half(), xs.cpu(), torch.ones(8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            moe.matmul_int(lin, xq, x_scale=sc)
    with pytest.raises(ValueError):
        moe.matmul_int(lin, x, x_scale=xs)
    for out in (torch.empty((4, 15), dtype=BF16, device="cuda"), torch.empty((4, 16), dtype=F32, device="cuda"),
                torch.empty((1, 16), dtype=BF16, device="cuda").expand(4, 16)):
        with pytest.raises(ValueError):
            moe.matmul_int(lin, x, out=out)
    with pytest.raises(ValueError):
        moe.matmul_int(lin, x, residual=normal(g, (4, 15), BF16))
    with pytest.raises(moe.MoeError):  # out over x
        moe.matmul_int(lin, x, out=x[:, :16])
    with pytest.raises(moe.MoeError) as e:
        moe.matmul_int(lin, x, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    w, s = codes(g, (16, 32)), torch.ones(16, device="cuda")
    for kw in (dict(w_scale=s[:15]), dict(w_scale=s.half()), dict(w=w.int()), dict(w=w.t()), dict(w=w[:1].expand(16, 32)),
               dict(w_up=w), dict(w_up=w[:8], w_up_scale=s), dict(bias=s[:5]), dict(bias=s.double()), dict(bias_up=s),
               dict(out_dtype=I8), dict(w=w[0]), dict(w_scale=s[:1].expand(16))):
        with pytest.raises(ValueError):
            moe.LinearInt.from_tensors(**{**dict(w=w, w_scale=s), **kw})
    el = make_linear(g, 4, 16, 32)
    _, plan = plan_of(routing(np.random.default_rng(0), 4, 4, 2), 4)
    for kw in (dict(rows="tokens"), dict(n_slots=9), dict(n_slots=-1), dict(top_k=0), dict(x=x[:3]), dict(rows="slot")):
        with pytest.raises(ValueError):
            moe.grouped_matmul_int(el, **{**dict(x=x, plan=plan, n_slots=8, top_k=2), **kw})
    for bad in (dict(codes=torch.empty((4, 32), device="cuda")), dict(codes=torch.empty((4, 31), dtype=I8, device="cuda")),
                dict(scales=torch.empty(3, device="cuda")), dict(scales=torch.empty(4, dtype=F16, device="cuda"))):
        with pytest.raises(ValueError):
            moe.quantize_rows(x, **bad)
    with pytest.raises(ValueError):
        moe.quantize_rows(x.double())
