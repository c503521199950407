"""The scored router at the ends of its range, against its definition in 64 bits: values whose differences
or sums pass fp32's largest number, chosen experts far below the others, and tokens next to ones whose
order 32 bits leave open (router_ref.py derives the tolerances)."""

import numpy as np
import pytest
import torch

import quantized_expert_gemv_moe_amd as moe
from gpu_helpers import log
from test_gpu_router import DTYPES, compare, gen, logits_of

pytestmark = pytest.mark.gpu


def spread(E, k, rng):
    """Rows of both signs whose span passes fp32's largest number: one to all but one expert low, values alike and not."""
    rows = []
    for low in sorted({1, k - 1, k, k + 1, E // 2, E - k, E - 1} & set(range(1, E))):
        for high_std, low_std in ((0.0, 0.0), (0.3, 0.0), (0.0, 0.3), (0.3, 0.3)):
            v = 2e38 * (1 + high_std * rng.uniform(-1, 1, E))
            at = rng.permutation(E)[:low]
            v[at] = -2e38 * (1 + low_std * rng.uniform(-1, 1, low))
            rows.append(v)
    one = rng.standard_normal(E)
    one[rng.integers(E)] = -3e38
    other = one.copy()
    other[(int(np.argmin(one)) + 1) % E] = 3e38
    return np.array(rows + [one, other])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep", [(2, 1, 1), (24, 1, 1), (24, 4, 2), (64, 1, 1), (256, 8, 3), (512, 16, 5), (500, 1, 1),
                                      (600, 1, 1), (640, 32, 7)])
def test_logits_whose_span_passes_the_largest_number(E, G, keep, score, dtype):
    log(f"[case] router span {E} {G} {keep} {score} {dtype}")
    rng = np.random.default_rng(E + G)
    for k in sorted({1, min(8, E // G * keep)}):
        logits = torch.tensor(spread(E, k, rng), device="cuda").to(DTYPES[dtype])
        assert bool(torch.isfinite(logits).all()) and bool((logits > torch.finfo(DTYPES[dtype]).min).all())
        for by, renorm in (("max", True), ("top2", False)):
            r = moe.Router(E, k, score=score, n_groups=G, top_groups=keep, group_score=by, renormalise=renorm)
            compare(logits, dtype, r, f"span E={E} G={G} k={k} {by}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep", [(2, 1, 1), (24, 4, 2), (256, 8, 3), (512, 16, 5), (600, 1, 1)])
def test_biases_whose_span_passes_the_largest_number(E, G, keep, score):
    log(f"[case] router bias span {E} {G} {keep} {score}")
    rng = np.random.default_rng(E)
    k = min(8, E // G * keep)
    logits = logits_of(E, 6, E, "fp32")
    for row in spread(E, k, rng):
        bias = torch.tensor(row, dtype=torch.float32, device="cuda")
        for by in ("max", "top2"):
            r = moe.Router(E, k, score=score, bias=bias, n_groups=G, top_groups=keep, group_score=by)
            compare(logits, "fp32", r, f"bias span E={E} G={G} {by}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_whose_sums_pass_the_largest_number(score):
    """Sums of two biases that fp32 holds and fp32 would make infinite, of either sign: groups in the order of the sums."""
    log(f"[case] router group sums {score}")
    pairs = {(2, 1): [[0, 0], [3.3e38, 0.3e38], [2.5e38, 2.5e38], [0, 0]],
             (2, 2): [[1.8e38, 1.7e38], [3.3e38, 0.3e38], [2.5e38, 2.5e38], [3.4e38, 3.4e38]],
             (2, 3): [[-3e38, -3e38], [-2e38, -2e38], [-3.2e38, -1e38], [-2.5e38, -2.5e38]]}
    for (per, keep), groups in pairs.items():
        for order in ((0, 1, 2, 3), (2, 1, 3, 0), (3, 2, 1, 0)):
            for wide in (1, 3, 16):  # two of a group's experts, the others far below
                bias = torch.full((4, per * wide), -3.3e38, device="cuda")
                for g, o in enumerate(order):
                    bias[g, [0, per * wide - 1]] = torch.tensor(groups[o], dtype=torch.float32, device="cuda")
                bias = bias.view(-1).contiguous()
                E = bias.numel()
                for k in {1, min(8, per * wide * keep)}:
                    r = moe.Router(E, k, score=score, bias=bias, n_groups=4, top_groups=keep, group_score="top2")
                    compare(logits_of(E, 5, E, "fp32"), "fp32", r, f"sums {order} E={E} keep={keep} k={k}")


@pytest.mark.parametrize("low", [0.0, -712.0, -730.0, -744.0, -800.0, -1e5, -2e38])
@pytest.mark.parametrize("E,G", [(64, 1), (256, 8), (600, 1), (640, 32)])
def test_renormalised_softmax_far_below_the_largest_logit(E, G, low):
    """The chosen experts' weights are the softmax of their own logits, however far an expert that the bias leaves out is
    above them, and whether 32 bits or the whole wave settle the token."""
    log(f"[case] router far below {E} {G} {low}")
    k, chosen = 6, np.arange(3, 9) + E // 2
    logits = np.full((5, E), low)
    steps = np.array([0.0, -0.5, -1.25, 0.75, -3.0, 0.25])
    logits[:, chosen] += steps * max(1.0, abs(low) * 2.0 ** -20)  # (a step that fp32 holds next to low)
    logits[:, 0] = 0.0
    logits[2, 1] = -np.inf                    # a masked one: the whole wave's way
    logits[3, chosen] = low                   # all alike
    logits[4, chosen[2]] = min(low * 1.1, low - 30.0)
    bias = torch.zeros(E, device="cuda")
    bias[torch.as_tensor(chosen)] = 2.0 + torch.arange(k, 0, -1, device="cuda") * 0.5
    lg = torch.tensor(logits, dtype=torch.float32, device="cuda")
    for by, scale in (("max", 1.0), ("top2", 2.5)):
        r = moe.Router(E, k, bias=bias, n_groups=G, top_groups=1, group_score=by, scale=scale)
        idx, w = moe.router_topk(r, lg)
        torch.cuda.synchronize()
        assert idx.cpu().tolist() == [chosen.tolist()] * 5
        l = lg.double().cpu().numpy()[:, chosen]
        e = np.exp(l - l.max(axis=1, keepdims=True))
        want = e / e.sum(axis=1, keepdims=True) * scale
        # 64 bits, 2^-48 of exponentials, sum and quotient, then one rounding to fp32
        off = np.abs(w.double().cpu().numpy() - want)
        assert (off <= want * (2.0 ** -24 + 2.0 ** -48) + 2.0 ** -150).all(), f"{by}: {w.cpu()} for {want}"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("renorm", [False, True])
def test_a_token_does_not_notice_its_neighbours(renorm, biased, score):
    """The same bits whether a token is alone, next to ordinary tokens or next to ones that 32 bits cannot order, and
    from either entry point."""
    log(f"[case] router neighbours renorm={renorm} biased={biased} {score}")
    for E, G, keep in ((64, 1, 1), (256, 8, 4), (512, 16, 3)):
        T = 400
        logits = logits_of(E, T, E, "fp32", 2.0)
        bias = torch.empty(E, device="cuda").normal_(0.0, 0.1, generator=gen(1)) if biased else None
        if biased:
            bias[5] = bias[9] = 3.0  # two that are chosen, in an order that equal scores leave to their ids
        r = moe.Router(E, 8, score=score, bias=bias, n_groups=G, top_groups=keep, group_score="top2", renormalise=renorm)
        alone = [moe.router_topk(r, logits[t:t + 1]) for t in range(T)]
        idx, w = torch.cat([a[0] for a in alone]), torch.cat([a[1] for a in alone])
        for every in (2, 3, 4):
            mixed = logits.clone()
            mixed[::every] = 0.0                # all alike: open to the end
            mixed[::every, 9] = mixed[::every, 5] = 4.0
            got = moe.router_topk(r, mixed)
            plan = moe.router_plan(r, mixed[:64])
            torch.cuda.synchronize()
            keeps = torch.arange(T, device="cuda") % every != 0
            for i, ww in ((got[0], got[1]), (torch.cat([plan[0], got[0][64:]]), torch.cat([plan[1], got[1][64:]]))):
                assert torch.equal(i[keeps], idx[keeps])
                off = (ww[keeps].view(torch.int32) != w[keeps].view(torch.int32)).sum().item()
                assert off == 0, f"E={E} every={every}: {off} weights differ"
        compare(mixed, "fp32", r, f"neighbours E={E}")


@pytest.mark.parametrize("E,G,keep", [(64, 1, 1), (256, 8, 4), (512, 1, 1), (512, 16, 5)])
def test_biased_softmax_in_steps_around_the_proof(E, G, keep):
    """Values s + b that lie 2e-8 to 2e-4 of the largest score apart, below and above what the 32-bit scores are good to:
    a total of 512 exponentials is off by some 40 of its last places where all of them round the same way."""
    log(f"[case] router biased softmax in steps {E} {G} {keep}")
    rng = np.random.default_rng(E + G)
    T, k = 96, 8
    b = torch.tensor(rng.uniform(-0.4, 0.4, E) / E, dtype=torch.float32, device="cuda")
    bias = b.double().cpu().numpy()
    rows = []
    for step in 2e-8 * 10.0 ** np.linspace(0, 4, T):
        c = (1.0 + bias.sum()) / E + np.where(rng.random(E) < 24 / E, step, -30 * step) / E * rng.permutation(E) * 24 / E
        rows.append(np.log(np.maximum(c - bias, 0.1 / E)) + rng.uniform(-8, 8))
    logits = torch.tensor(np.array(rows), dtype=torch.float32, device="cuda")
    for by in ("max", "top2"):
        for renorm in (True, False):
            r = moe.Router(E, k, bias=b, n_groups=G, top_groups=keep, group_score=by, renormalise=renorm)
            compare(logits, "fp32", r, f"steps E={E} G={G} {by}")


@pytest.mark.parametrize("E,G,keep", [(24, 1, 1), (256, 8, 3), (512, 16, 5), (600, 1, 1), (640, 32, 7)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_logit_that_only_a_bias_masks(value, E, G, keep):
    """It is in the sum of every softmax score, so the token has no numbers; a sigmoid's other scores know nothing of it.
    One that its logit masks as well counts for nothing."""
    log(f"[case] router masked by bias, logit {value}, {E} {G} {keep}")
    k, at = 5, E // 2 + 1
    logits = logits_of(E, 9, E, "fp32")
    bias = torch.empty(E, device="cuda").normal_(0.0, 0.1, generator=gen(2))
    bias[at] = -float("inf")
    other = logits.clone()
    other[[2, 5], at] = value
    other[4, at] = -float("inf")
    for by in ("max", "top2"):
        for renorm in (True, False):
            kw = dict(bias=bias, n_groups=G, top_groups=keep, group_score=by, renormalise=renorm)
            r = moe.Router(E, k, score="sigmoid", **kw)
            want, got = moe.router_topk(r, logits), moe.router_topk(r, other)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not bool((got[0] == at).any())
            r = moe.Router(E, k, score="softmax", **kw)
            idx, w = moe.router_topk(r, other)
            torch.cuda.synchronize()
            assert bool((idx[[2, 5]] == -1).all()) and bool(torch.isnan(w[[2, 5]]).all())
            rest = [0, 1, 3, 4, 6, 7, 8]
            compare(other[rest], "fp32", r, f"beside them {by} {renorm}", got=(idx[rest], w[rest]))
