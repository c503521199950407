"""Uses of the products that their documentation allows: plans and workspaces kept between
batches, halves of one stack per expert, single rows and columns in strided buffers, streams and
graphs around the split over K."""

import numpy as np
import pytest
import torch

import matmul_ref as ref
import quantized_expert_gemv_moe_amd as moe
from gpu_helpers import log
from test_gpu_matmul import gen, make_linear, normal, plan_of, reference, routing

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def check_rows(lin, x, idx, out, rows, act, tag):
    """out of a grouped product by slot or token against the definition, slots of no expert apart."""
    flat, k = idx.reshape(-1), idx.shape[1]
    for e in range(lin.n_groups):
        mine = torch.nonzero(flat == e)[:, 0]
        if mine.numel():
            src = mine // k if rows == "token" else mine
            ref.check(out[mine], *reference(lin, act, 0.0, x[src], e=e), f"{tag} e={e}")


def test_a_plan_and_a_workspace_for_batches_of_falling_size():
    """Buffers for the largest batch, used for it first and then for smaller ones: nothing of
    an earlier batch is seen in a later one."""
    g = gen(61)
    E, k, K, N = 6, 2, 8192, 64  # K goes in stretches
    lin = make_linear(g, E, N, K, BF16, True, True, "silu", BF16)
    plan = moe.Plan.allocate(E, 300 * k)
    ws = moe.alloc_grouped_workspace(lin, 300 * k)
    for T in (300, 40, 7, 2, 1, 90):
        log(f"[case] falling sizes T={T}")
        idx = torch.as_tensor(routing(np.random.default_rng(T), T, E - 2, k)).cuda()
        moe.expert_plan(idx, E, plan=plan)
        x = normal(g, (T, K), BF16)
        out = moe.grouped_matmul(lin, x, plan, T * k, top_k=k, workspace=ws)
        torch.cuda.synchronize()
        check_rows(lin, x, idx, out, "token", "silu", f"T={T}")


@pytest.mark.parametrize("T", [3, 60, 900])
def test_grouped_halves_of_one_stack(T):
    """gate and up, and their biases, as halves of one stack per expert."""
    log(f"[case] halves T={T}")
    g = gen(62)
    E, k, K, N = 5, 2, 320, 72
    w, b = normal(g, (E, 2 * N, K), BF16, 0.05), normal(g, (E, 2 * N), BF16, 0.5)
    lin = moe.Linear.from_tensors(w[:, :N], w_up=w[:, N:], bias=b[:, :N], bias_up=b[:, N:], activation="silu")
    idx, plan = plan_of(routing(np.random.default_rng(T), T, E, k), E)
    x = normal(g, (T, K), BF16)
    out = moe.grouped_matmul(lin, x, plan, T * k, top_k=k)
    torch.cuda.synchronize()
    check_rows(lin, x, idx, out, "token", "silu", f"T={T}")


def test_single_columns_and_rows_of_wider_buffers():
    """K of one and N of one, whose strides are those of the buffers they were cut from."""
    g = gen(63)
    w, x, o = normal(g, (40, 9), F32), normal(g, (30, 7), F32), torch.zeros((30, 50), device="cuda")
    lin = moe.Linear.from_tensors(w[:, 3:4])
    moe.matmul(lin, x[:, 2:3], out=o[:, :40])
    ref.check(o[:, :40], *ref.product(x[:, 2:3], w[:, 3:4]), "K of one")
    assert bool((o[:, 40:] == 0).all())
    lin = moe.Linear.from_tensors(w[5:6, :7])
    moe.matmul(lin, x, out=o[:, 44:45])
    torch.cuda.synchronize()
    ref.check(o[:, 44:45], *ref.product(x, w[5:6, :7]), "N of one")
    assert bool((o[:, 45:] == 0).all()) and bool((o[:, 40:44] == 0).all())
    we = normal(g, (4, 3, 64), BF16)
    el = moe.Linear.from_tensors(we[:, 1:2])  # experts of one column, three rows apart
    idx, plan = plan_of(np.arange(8, dtype=np.int32).reshape(8, 1) % 4, 4)
    xe = normal(g, (8, 64), BF16)
    check_rows(el, xe, idx, moe.grouped_matmul(el, xe, plan, 8), "slot", "none", "N of one per expert")
    one = moe.Linear.from_tensors(we[:1])
    idx, plan = plan_of(np.zeros((8, 1), np.int32), 1)
    check_rows(one, xe, idx, moe.grouped_matmul(one, xe, plan, 8), "slot", "none", "one expert")
    ref.check(moe.matmul(one, xe), *ref.product(xe, we[0], out_dtype=BF16), "one expert, dense")


def test_split_products_in_graphs():
    """The two launches of the split over K, captured with a workspace that the call allocates and
    with one each of the caller's; replays in turn with eager calls between."""
    g = gen(64)
    lin = make_linear(g, None, 512, 8192, BF16, False, True, "silu", BF16)
    assert moe.matmul_workspace_size(lin, 64) > 0
    graphs = []
    for own in (False, True, True):
        x, out = normal(g, (64, 8192), BF16), torch.empty((64, 512), dtype=BF16, device="cuda")
        ws = moe.alloc_matmul_workspace(lin, 64) if own else None
        moe.matmul(lin, x, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.matmul(lin, x, out=out, workspace=ws)
        graphs.append((graph, x, out, ws))
    for i in range(4):
        for graph, x, out, ws in graphs:
            x.copy_(normal(g, x.shape, BF16))
            want = moe.matmul(lin, x)
            out.fill_(float("nan"))
            if ws is not None:
                ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), f"replay {i}"
    ref.check(want, *reference(lin, "silu", 0.0, graphs[-1][1]), "split")


def test_grouped_and_combine_on_other_streams():
    g = gen(65)
    E, k, T, K, N = 4, 2, 50, 4096, 96
    lin = make_linear(g, E, N, K, BF16, False, False, "none", F32)
    idx, plan = plan_of(routing(np.random.default_rng(3), T, E, k), E)
    w = torch.softmax(normal(g, (T, k), F32), dim=1)
    x = normal(g, (T, K), BF16)
    want = moe.combine(moe.grouped_matmul(lin, x, plan, T * k, top_k=k), idx, w, E)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams * 3:
        y = moe.grouped_matmul(lin, x, plan, T * k, top_k=k, stream=s)
        outs.append(moe.combine(y, idx, w, E, stream=s))
        with torch.cuda.stream(s):
            outs.append(moe.combine(moe.grouped_matmul(lin, x, plan, T * k, top_k=k), idx, w, E))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_combine_of_no_tokens_and_of_zero_weights():
    g = gen(66)
    none = moe.combine(torch.empty((0, 16), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                       torch.empty((0, 2), device="cuda"), 4, out_dtype=BF16)
    assert none.shape == (0, 16) and none.dtype == BF16
    idx, y, r = torch.zeros((5, 3), dtype=torch.int32, device="cuda"), normal(g, (15, 20), F32), normal(g, (5, 20), F32)
    out = moe.combine(y, idx, torch.zeros((5, 3), device="cuda"), 4, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(out, r)
