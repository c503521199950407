"""Every kernel of the integer products, in both forms, dense and per expert, against 64 bits: ordinary
and odd outputs, strides and addresses; calls next to one another; and the calls that a model makes of
them over and over (int_ref.py derives the tolerances)."""

import numpy as np
import pytest
import torch

import int_cases
import int_ref as ref
import quantized_expert_gemv_moe_amd as moe
from gpu_helpers import log
from test_gpu_matmul_int import (BF16, F16, F32, I8, SENTINEL, codes, gen, make_linear, make_x, normal, out_view, plan_of,
                                 reference, routing, strided)

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": F32, "bf16": BF16, "fp16": F16, "int8": I8}
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


def case_id(c):
    return "-".join(map(str, c[:8]))


def workspace(nbytes, size):
    return torch.empty(size if nbytes < 0 else nbytes, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("n,case", [p for p in enumerate(int_cases.CASES) if p[1][3] == 0],
                         ids=lambda v: case_id(v) if isinstance(v, tuple) else str(v))
def test_dense_kernels(n, case):
    xt, ot, gated, _, rows, _, K, N, off, ws, kernel = case
    g = gen(n)
    # functions, biases, residuals and outputs: usual ones, then strange ones
    for i, (act, bias, res, pad, o_off) in enumerate(((ACTS[n % 2], None, ot, 0, 0), (ACTS[n % 3 + 2], F32, "fp32", 3, 1),
                                                      (ACTS[(n + 1) % 5], F16, "bf16", 8, 2), ("silu", BF16, None, 5, 3))):
        log(f"[case] int kernel {kernel} {case[:9]} act={act} bias={bias} residual={res} pad={pad} at={o_off}")
        lin = make_linear(g, None, N, K, gated, bias, act, DTYPES[ot], 1.5 if i == 2 else 0.0)
        x0, xs, q, s = make_x(g, rows, K, DTYPES[xt])
        x = strided(x0, 0, off)
        residual = None if res is None else strided(normal(g, (rows, N), DTYPES[res]), pad, o_off)
        out, untouched = out_view(rows, N, DTYPES[ot], pad, o_off)
        moe.matmul_int(lin, x, x_scale=xs, residual=residual, out=out,
                       workspace=workspace(ws, moe.matmul_int_workspace_size(lin, rows)))
        torch.cuda.synchronize()
        ref.check(out, *reference(lin, act, 1.5 if i == 2 else 0.0, q, s, residual), f"{case_id(case)} {i}")
        untouched()


@pytest.mark.parametrize("rows", ["slot", "token", "sorted"])
@pytest.mark.parametrize("n,case", [p for p in enumerate(int_cases.CASES) if p[1][3] > 0],
                         ids=lambda v: case_id(v) if isinstance(v, tuple) else str(v))
def test_expert_kernels(n, case, rows):
    xt, ot, gated, E, T, k, K, N, off, ws, kernel = case
    g = gen(n)
    idx = routing(np.random.default_rng(n), T, E, k, 0.5)
    if T > 2:
        idx[T // 2, 0] = -1  # a slot that no expert computes
    flat = idx.reshape(-1)
    total = T * k
    _, plan = plan_of(idx, E)
    for i, (act, bias, pad, o_off) in enumerate(((ACTS[n % 2], None, 0, 0), (ACTS[(n + 2) % 5], BF16, 3, 1))):
        log(f"[case] int expert kernel {kernel} {case[:9]} rows={rows} act={act} bias={bias} pad={pad} at={o_off}")
        lin = make_linear(g, E, N, K, gated, bias, act, DTYPES[ot])
        x_rows = T if rows == "token" else total
        x0, xs, q, s = make_x(g, x_rows, K, DTYPES[xt])
        x = strided(x0, 0, off)
        out, untouched = out_view(total, N, DTYPES[ot], pad, o_off)
        moe.grouped_matmul_int(lin, x, plan, total, top_k=k, rows=rows, x_scale=xs, out=out,
                               workspace=workspace(ws, moe.grouped_int_workspace_size(lin, total, x_rows)))
        torch.cuda.synchronize()
        want = torch.full((total, N), SENTINEL, dtype=DTYPES[ot], device="cuda").double()
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
            want[dst], tol[dst] = reference(lin, act, 0.0, q[src], s[src], e=e)
        ref.check(out, want, tol, f"{case_id(case)} {rows} {i}")
        untouched()


@pytest.mark.parametrize("rows,K,N,dtype", [(4486, 176, 876, BF16), (5986, 1088, 2094, F32), (5986, 1088, 2096, F16),
                                            (4486, 176, 100, BF16)])
def test_large_tiles_over_their_residual(rows, K, N, dtype):
    """Columns of the last tile that the tile before has too must not have the residual added twice."""
    log(f"[case] large in place {rows} {K} {N} {dtype}")
    g = gen(N)
    lin = make_linear(g, None, N, K, False, BF16, "gelu", dtype)
    x, xs, q, s = make_x(g, rows, K, I8)
    out, untouched = out_view(rows, N, dtype, 3, 1)
    out.copy_(normal(g, (rows, N), dtype))
    kept = out.clone()
    apart = moe.matmul_int(lin, x, x_scale=xs, residual=kept)
    moe.matmul_int(lin, x, x_scale=xs, residual=out, out=out)
    torch.cuda.synchronize()
    ref.check(out, *reference(lin, "gelu", 0.0, q, s, kept), f"in place {rows} {N}")
    # (the last columns are finished by other code where out is the residual, and a compiler may fuse the last product
    # with the residual's sum in one and not in the other: one rounding, u |f|, which the tolerance counts)
    ref.check(apart, *reference(lin, "gelu", 0.0, q, s, kept), f"apart {rows} {N}")
    untouched()


@pytest.mark.parametrize("rows,K,N", [(1, 1003, 64), (300, 1003, 200), (1500, 333, 640), (4100, 1003, 1030)])
def test_integers_at_odd_addresses(rows, K, N):
    """Copied into the workspace or not, the sums are the same whole numbers: bit for bit one result where the function is
    none."""
    log(f"[case] odd integers {rows} {K} {N}")
    g = gen(rows)
    lin = make_linear(g, None, N, K, False, BF16, "none", BF16)
    x, xs, _, _ = make_x(g, rows, K, I8)
    wide = torch.zeros((rows, (K + 15) // 16 * 16), dtype=I8, device="cuda")
    wide[:, :K] = x
    want = moe.matmul_int(lin, wide[:, :K], x_scale=xs)
    for off in (0, 1, 8):
        for space in (None, torch.empty(256, dtype=torch.uint8, device="cuda")):
            got = moe.matmul_int(lin, strided(x, 0, off), x_scale=xs, workspace=space)
            torch.cuda.synchronize()
            assert torch.equal(got.view(torch.int16), want.view(torch.int16)), (off, space is None)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65])
@pytest.mark.parametrize("E,k,G,keep", [(256, 8, 8, 4), (160, 6, 8, 3), (132, 4, 4, 2), (512, 10, 16, 3), (513, 3, 1, 1),
                                        (640, 8, 32, 5), (64, 16, 1, 1), (300, 7, 1, 1)])
def test_router_and_plan_in_one_launch_and_two(E, k, G, keep, T):
    """Ids, weights and every record of the plan are those of the router and the planner one after the other."""
    log(f"[case] router and plan {E} {k} {G} {keep} T={T}")
    g = gen(E + T)
    logits = normal(g, (T, E), BF16)
    router = moe.Router(E, k, score="sigmoid", bias=normal(g, (E,), F32, 0.1), n_groups=G, top_groups=keep, group_score="top2")
    if T > 2:
        logits[1, 3] = float("nan")
        logits[2] = float("-inf")
    idx, w = moe.router_topk(router, logits)
    want = moe.expert_plan(idx, E)
    got_idx, got_w, plan = moe.router_plan(router, logits)
    torch.cuda.synchronize()
    assert torch.equal(got_idx, idx) and torch.equal(got_w.view(torch.int32), w.view(torch.int32))
    n = int(want.offsets[E])
    for name in ("counts", "offsets", "unique_experts", "n_unique", "work"):
        assert torch.equal(getattr(plan, name), getattr(want, name)), name
    assert torch.equal(plan.sorted_slots[:n], want.sorted_slots[:n])


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own, the same weights and rows: neither disturbs the other."""
    log("[case] int two at once")
    g = gen(5)
    for rows, K, N in ((300, 2048, 768), (40, 16384, 96), (2000, 1003, 1024)):
        lin = make_linear(g, None, N, K, True, BF16, "silu", BF16)
        xs = [normal(g, (rows, K), BF16) for _ in range(2)]
        want = [moe.matmul_int(lin, x) for x in xs]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        spaces = [moe.alloc_matmul_int_workspace(lin, rows) for _ in range(2)]
        outs = [torch.empty_like(want[0]) for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(8):
            for i in range(2):
                moe.matmul_int(lin, xs[i], out=outs[i], workspace=spaces[i], stream=streams[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i].view(torch.int16), want[i].view(torch.int16))


def test_many_shapes_in_one_graph():
    """Products of every launch form one after another in one graph, with one workspace (they run in their
    order); replayed on new inputs with eager work between."""
    log("[case] int one graph")
    g = gen(6)
    shapes = [(1, 512, 96, BF16), (40, 512, 96, BF16), (700, 256, 130, F32), (20, 16384, 64, BF16), (600, 333, 70, I8)]
    calls = []
    for rows, K, N, dt in shapes:
        lin = make_linear(g, None, N, K, True, BF16, "silu", BF16)
        x, s, _, _ = make_x(g, rows, K, dt)
        calls.append((lin, x, s, torch.empty((rows, N), dtype=BF16, device="cuda")))
    space = torch.empty(max(moe.matmul_int_workspace_size(c[0], c[1].shape[0]) for c in calls), dtype=torch.uint8, device="cuda")

    def run(outs):
        for (lin, x, s, _), o in zip(calls, outs):
            moe.matmul_int(lin, x, x_scale=s, out=o, workspace=space)

    run([c[3] for c in calls])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run([c[3] for c in calls])
    for i in range(3):
        for lin, x, s, o in calls:
            x.copy_(codes(g, x.shape) if x.dtype is I8 else normal(g, x.shape, x.dtype))
            o.fill_(float("nan"))
        eager = [torch.empty_like(c[3]) for c in calls]
        run(eager)
        graph.replay()
        torch.cuda.synchronize()
        for (_, _, _, o), e in zip(calls, eager):
            assert torch.equal(o.view(torch.int16), e.view(torch.int16)), f"replay {i}"


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [8, 17, 130, 512, 520, 1500, 4100])
def test_quantize_many_short_rows(cols, dtype):
    """The divisions of a block that take over from 4096 rows on, and the row before."""
    for rows in (4095, 4096, 4099):
        log(f"[case] quantize rows={rows} cols={cols} {dtype}")
        g = gen(rows + cols)
        x = normal(g, (rows, cols), dtype)
        x[7], x[11, 0], x[rows - 1, cols - 1] = 0, float("nan"), float("inf")
        q, s = moe.quantize_rows(x)
        torch.cuda.synchronize()
        want_q, want_s = ref.quantize(x)
        assert torch.equal(q.double(), want_q)
        assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(want_s, nan=-1.0))
