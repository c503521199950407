"""moe_router_topk and moe_router_plan on the GPU against their definition in 64 bits
(router_ref.py derives the tolerances)."""

import numpy as np
import pytest
import torch

import quantized_expert_gemv_moe_amd as moe
import router_ref
from gpu_helpers import log

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def logits_of(seed, T, E, dtype, std=1.0):
    return torch.empty((T, E), device="cuda").normal_(0.0, std, generator=gen(seed)).to(DTYPES[dtype])


def compare(logits, dtype, router, tag, got=None):
    idx, w = moe.router_topk(router, logits) if got is None else got
    torch.cuda.synchronize()
    bias = None if router.bias is None else router.bias.double().cpu().numpy()
    ids, want, tol = router_ref.route(logits.double().cpu().numpy(), dtype, router.top_k, router.score, bias,
                                      router.n_groups, router.top_groups, router.group_score, router.renormalise,
                                      router.scale)
    idx, w = idx.cpu().numpy(), w.double().cpu().numpy()
    bad = np.nonzero((idx != ids).any(axis=1))[0]
    assert bad.size == 0, f"{tag}: token {bad[0]}: {idx[bad[0]]} for {ids[bad[0]]} ({bad.size} tokens)"
    assert np.array_equal(np.isnan(w), np.isnan(want)), f"{tag}: NaN in other places"
    live = ~np.isnan(want)
    off = np.abs(w - want)[live] > tol[live]
    assert not off.any(), f"{tag}: {int(off.sum())} weights off, worst {np.abs(w - want)[live].max()}"
    return ids


# tokens, experts, top_k, groups, kept
SHAPES = [(1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (2, 3, 3, 1, 1), (3, 60, 4, 1, 1), (5, 64, 16, 1, 1), (17, 65, 6, 1, 1),
          (33, 128, 8, 1, 1), (9, 128, 8, 4, 2), (40, 160, 6, 8, 3), (7, 100, 5, 10, 3), (12, 120, 7, 8, 2),
          (6, 257, 8, 1, 1), (8, 512, 8, 16, 5), (4, 1000, 9, 8, 2), (3, 1024, 16, 1, 1), (5, 1024, 8, 64, 9),
          (4, 1020, 8, 5, 2), (6, 1023, 5, 33, 4), (11, 6, 2, 6, 4), (10, 30, 2, 15, 1), (100, 96, 8, 3, 3)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_router_shapes(shape, biased, score, dtype):
    T, E, k, G, keep = shape
    log(f"[case] router {shape} biased={biased} {score} {dtype}")
    logits = logits_of(T + E, T, E, dtype, 2.0)
    bias = torch.empty(E, device="cuda").normal_(0.0, 0.2, generator=gen(E)) if biased else None
    for by, renorm, scale in (("max", True, 1.0), ("top2", True, 2.5), ("max", False, 0.5), ("top2", False, 1.0)):
        r = moe.Router(E, k, score=score, bias=bias, n_groups=G, top_groups=keep, group_score=by, renormalise=renorm,
                       scale=scale)
        compare(logits, dtype, r, f"{shape} {score} {dtype} biased={biased} {by} renorm={renorm}")


def test_many_tokens_keep_the_exact_order():
    """Scores next to one another: 32 bits would put some of these tokens' experts in another order."""
    T, E, k = 6000, 256, 8
    log("[case] router many tokens")
    for score, dtype in (("sigmoid", "fp32"), ("softmax", "fp32"), ("sigmoid", "bf16")):
        logits = logits_of(5, T, E, dtype, 0.05)
        bias = torch.empty(E, device="cuda").normal_(0.0, 0.001, generator=gen(6))
        r = moe.Router(E, k, score=score, bias=bias, n_groups=8, top_groups=4, group_score="top2", scale=2.5)
        compare(logits, dtype, r, f"many {score} {dtype}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_clusters_of_close_values(score, biased):
    """Values closer than 32 bits or a 22-bit place in their range can tell apart: a few among the
    chosen, at the border, more than are looked at again, groups next to one another, and one far
    value that widens the range."""
    log(f"[case] router clusters {score} biased={biased}")
    for E, G, keep in ((256, 1, 1), (256, 8, 4), (64, 1, 1), (512, 16, 3), (40, 1, 1), (16, 1, 1)):
        rng = np.random.default_rng(E + G)
        rows = []
        for size in (2, 3, 8, 9, 12, 20, E):
            for step in (2.0 ** -23, 2.0 ** -21, 1e-5):
                v = rng.standard_normal(E) * 0.3
                at = rng.permutation(E)[:min(size, E)]
                v[at] = 1.0 + step * rng.permutation(at.size)
                rows.append(v)
                far = v.copy()
                far[rng.integers(E)] = rng.choice([1e4, -1e4])
                rows.append(far)
        one = rng.standard_normal(E // G)
        rows += [np.tile(one, G) + 1e-7 * rng.standard_normal(E), np.tile(one, G)]
        logits = torch.tensor(np.array(rows), dtype=torch.float32, device="cuda")
        bias = torch.tensor((rng.integers(0, 3, E) - 1) * 2.0 ** -20, dtype=torch.float32, device="cuda") if biased else None
        for by in ("max", "top2"):
            for k in (2, 8, 15, 16):
                r = moe.Router(E, k, score=score, bias=bias, n_groups=G, top_groups=keep, group_score=by)
                compare(logits, "fp32", r, f"clusters {E} {G} {by} k={k}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_ties_go_to_the_lower_expert_and_group(score, biased):
    log(f"[case] router ties {score} biased={biased}")
    for E, G, keep in ((64, 1, 1), (256, 8, 3), (160, 8, 2), (1020, 5, 2)):
        rng = np.random.default_rng(E)
        rows = [np.zeros(E), np.full(E, -5.0), rng.integers(0, 2, E).astype(float), rng.integers(-2, 3, E) * 0.5,
                np.where(np.arange(E) % 7 == 3, 1.0, 0.0), -np.zeros(E) * (np.arange(E) % 2), np.full(E, 30.0)]
        logits = torch.tensor(np.array(rows), dtype=torch.float32, device="cuda")
        bias = torch.tensor((np.arange(E) % 3) * 0.25, dtype=torch.float32, device="cuda") if biased else None
        for by in ("max", "top2"):
            r = moe.Router(E, 8, score=score, bias=bias, n_groups=G, top_groups=keep, group_score=by)
            compare(logits, "fp32", r, f"ties {E} {G} {by}")


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_masks_infinities_and_nan(biased, score, dtype):
    """Masked experts are chosen last and weigh nothing; a token whose scores are not numbers has
    ids -1 and weights NaN, and no other token notices."""
    low = router_ref.LOWEST[dtype]
    inf, nan = float("inf"), float("nan")
    log(f"[case] router masks {score} biased={biased} {dtype}")
    for E, G, keep, k in ((24, 1, 1, 8), (24, 4, 2, 8), (130, 1, 1, 8), (256, 8, 2, 8)):
        rng = np.random.default_rng(E + G)
        base = rng.standard_normal((16, E)) * 2
        base[1, :] = -inf                                   # nothing left
        base[2, :] = low
        base[3, rng.permutation(E)[:E - 3]] = -inf          # fewer than k left
        base[4, rng.permutation(E)[:E - 1]] = low
        base[5, :E // 2] = -inf
        base[6, E // 2:] = low
        base[7, 5] = nan
        base[8, 0] = inf
        base[9, :] = nan
        base[10, 3], base[10, 4] = inf, -inf
        base[11, :] = inf
        base[12, E - 1], base[12, 0] = nan, -inf
        base[13, ::2] = -inf
        base[14, :] = 0.99 * low                            # low, but not masked
        logits = torch.tensor(base, dtype=torch.float32, device="cuda").to(DTYPES[dtype])
        assert bool((logits[2] == torch.finfo(DTYPES[dtype]).min).all()) and bool(torch.isfinite(logits[14]).all())
        bias = torch.tensor(rng.standard_normal(E) * 0.1, dtype=torch.float32, device="cuda") if biased else None
        for by, renorm in (("max", True), ("top2", True), ("top2", False)):
            r = moe.Router(E, k, score=score, bias=bias, n_groups=G, top_groups=keep, group_score=by, renormalise=renorm)
            compare(logits, dtype, r, f"masks E={E} G={G} {by} {renorm}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_are_not_finite(score):
    log(f"[case] router biases {score}")
    E, inf, nan = 40, float("inf"), float("nan")
    logits = logits_of(8, 6, E, "fp32")
    logits[2, 7] = -inf
    for at, v in ((7, -inf), (7, inf), (7, nan)):
        bias = torch.zeros(E, device="cuda")
        bias[at] = v
        for k in (5, 16):
            compare(logits, "fp32", moe.Router(E, k, score=score, bias=bias), f"bias[{at}]={v} k={k}")
    bias = torch.full((E,), -inf, device="cuda")
    bias[[3, 9]] = 0.5
    compare(logits, "fp32", moe.Router(E, 4, score=score, bias=bias), "all but two masked by bias")


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_strided_logits_and_given_outputs(dtype):
    """Rows apart and at any element; nothing else is read or written."""
    log(f"[case] router strides {dtype}")
    for T, E, pad, offset in ((5, 60, 3, 1), (21, 256, 5, 3), (9, 128, 128, 0), (300, 65, 1, 7)):
        buf = torch.full((offset + T * (E + pad) + 64,), float("nan"), dtype=DTYPES[dtype], device="cuda")
        view = buf[offset:offset + T * (E + pad)].view(T, E + pad)[:, :E]
        view.copy_(logits_of(T, T, E, dtype))
        store_i = torch.full((T * 6 + 32,), 77, dtype=torch.int32, device="cuda")
        store_w = torch.full((T * 6 + 32,), 77.0, device="cuda")
        idx, w = store_i[16:16 + T * 6].view(T, 6), store_w[16:16 + T * 6].view(T, 6)
        r = moe.Router(E, 6, score="sigmoid")
        got = moe.router_topk(r, view, idx=idx, w=w)
        assert got[0] is idx and got[1] is w
        compare(view, dtype, r, f"strides {T}x{E}+{pad}", got=got)
        for s in (store_i, store_w):
            assert bool((s[:16] == 77).all()) and bool((s[16 + T * 6:] == 77).all())


def test_rows_past_4_gib():
    log("[case] router far rows")
    T, E, stride = 520, 64, 1 << 22
    buf = torch.empty((T, stride), dtype=torch.bfloat16, device="cuda")
    view = buf[:, :E]
    view.copy_(logits_of(3, T, E, "bf16"))
    compare(view, "bf16", moe.Router(E, 4), "far rows")


@pytest.mark.parametrize("T", [0, 1, 2, 8, 9, 16, 17, 40, 300])
@pytest.mark.parametrize("E,k,G,keep", [(60, 4, 1, 1), (256, 8, 8, 4), (1024, 16, 1, 1), (1020, 8, 5, 2), (5, 5, 1, 1)])
def test_router_plan(E, k, G, keep, T):
    """The router's choice and the planner's plan of it, from one call; a token without numbers is
    left out of the plan."""
    log(f"[case] router plan T={T} E={E}")
    logits = logits_of(T + 1, T, E, "fp32")
    if T > 2:
        logits[1, 2] = float("nan")
    bias = torch.empty(E, device="cuda").normal_(0.0, 0.1, generator=gen(4))
    r = moe.Router(E, k, score="sigmoid", bias=bias, n_groups=G, top_groups=keep, group_score="top2")
    idx, w, plan = moe.router_plan(r, logits)
    want = moe.expert_plan(idx, E)
    one = moe.router_topk(r, logits)
    torch.cuda.synchronize()
    if T:
        compare(logits, "fp32", r, f"plan T={T} E={E}", got=(idx, w))
    assert torch.equal(idx, one[0]) and torch.equal(w.view(torch.int32), one[1].view(torch.int32))
    n = int(want.offsets[-1].item())
    assert n == k * (T - (T > 2))
    for name in ("counts", "offsets", "unique_experts", "n_unique", "work"):
        assert torch.equal(getattr(plan, name), getattr(want, name)), name
    assert torch.equal(plan.sorted_slots[:n], want.sorted_slots[:n])


def test_softmax_renormalised_is_the_plain_router():
    log("[case] router against route_topk")
    for T, E, k in ((1, 128, 8), (50, 128, 8), (33, 300, 6)):
        logits = logits_of(T, T, E, "fp32")
        idx, w = moe.route_topk(logits, k)
        got_idx, got_w = moe.router_topk(moe.Router(E, k), logits)
        torch.cuda.synchronize()
        assert torch.equal(idx, got_idx)
        assert float((w - got_w).abs().max()) <= 1e-6


def test_no_tokens():
    idx, w = moe.router_topk(moe.Router(8, 2), torch.empty((0, 8), device="cuda"))
    assert idx.shape == (0, 2) and w.shape == (0, 2)


def test_other_streams_and_a_graph():
    """On the caller's stream, and captured and replayed on new logits, twice the same graph's
    buffers with eager calls between."""
    log("[case] router streams and graphs")
    E, k, T = 256, 8, 12
    bias = torch.empty(E, device="cuda").normal_(0.0, 0.1, generator=gen(1))
    r = moe.Router(E, k, score="sigmoid", bias=bias, n_groups=8, top_groups=4, group_score="top2")
    big = logits_of(2, 500, E, "bf16")
    want = moe.router_topk(r, big)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [moe.router_topk(r, big, stream=side), moe.router_topk(r, big)]
    with torch.cuda.stream(side):
        outs.append(moe.router_topk(r, big))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    logits = logits_of(3, T, E, "fp32")
    plan = moe.Plan.allocate(E, T * k)
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    moe.router_plan(r, logits, plan=plan, idx=idx, w=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.router_plan(r, logits, plan=plan, idx=idx, w=w)
    for i in range(4):
        logits.copy_(logits_of(10 + i, T, E, "fp32"))
        eager = moe.router_plan(r, logits)
        idx.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, eager[0]) and torch.equal(w, eager[1])
        for name in ("counts", "offsets", "sorted_slots", "unique_experts", "n_unique", "work"):
            assert torch.equal(getattr(plan, name), getattr(eager[2], name)), name


def test_routed_quantised_layer():
    """The router's choice through the 4-bit expert block: what decode_step makes of the same ids and
    weights; a token whose logits are not numbers becomes NaN, the others are as without it."""
    from gpu_helpers import dev_x
    from moe_workloads import SHAPES, make_layer, make_x

    log("[case] router with the quantised layer")
    sh = SHAPES["toy"]
    L = make_layer(sh, experts=np.arange(sh.n_experts), seed=0)
    dl = moe.DeviceLayer.from_host(L)
    x = dev_x(make_x(sh, 5, seed=1))
    logits = logits_of(9, 5, sh.n_experts, "fp32")
    r = moe.Router(sh.n_experts, sh.top_k, score="sigmoid", scale=1.5)
    idx, w, plan = moe.router_plan(r, logits)
    out = moe.decode_step(dl, x, idx, w, plan)
    bad = logits.clone()
    bad[3, 0] = float("nan")
    idx2, w2, plan2 = moe.router_plan(r, bad)
    out2 = moe.decode_step(dl, x, idx2, w2, plan2)
    torch.cuda.synchronize()
    compare(logits, "fp32", r, "with the layer", got=(idx, w))
    rows = [0, 1, 2, 4]
    assert bool(torch.isnan(out2[3]).all()) and torch.equal(out[rows], out2[rows])
    assert bool(torch.isfinite(out.float()).all())


def test_wrappers_refuse_what_does_not_fit():
    r = moe.Router(8, 2)
    lg = torch.zeros((3, 8), device="cuda")
    for bad in (lg[:, :7], lg.double(), lg.cpu(), lg.t(), lg[:1].expand(3, 8), lg[0]):
        with pytest.raises(ValueError):
            moe.router_topk(r, bad)
    i32 = torch.int32
    for idx in (torch.empty((3, 3), dtype=i32, device="cuda"), torch.empty((3, 2), device="cuda"),
                torch.empty((3, 2), dtype=i32), torch.empty((2, 3), dtype=i32, device="cuda").t()):
        with pytest.raises(ValueError):
            moe.router_topk(r, lg, idx=idx)
    for w in (torch.empty((3, 2), dtype=torch.float16, device="cuda"), torch.empty((2, 2), device="cuda")):
        with pytest.raises(ValueError):
            moe.router_topk(r, lg, w=w)
    with pytest.raises(ValueError):
        moe.router_plan(r, lg, plan=moe.Plan.allocate(8, 5))
    with pytest.raises(moe.MoeError):  # outputs over the logits
        moe.router_topk(r, lg, w=lg.view(-1)[:6].view(3, 2))
    for bias in (torch.zeros(7, device="cuda"), torch.zeros(8, device="cuda", dtype=torch.bfloat16),
                 torch.zeros(16, device="cuda")[::2]):
        with pytest.raises(ValueError):
            moe.Router(8, 2, bias=bias)
