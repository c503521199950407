"""The scored router token by token in 64 bits, as moe_router_t defines it, and how far an
evaluation in fp32 and fp64 with one rounding may be from its weights.

Ids are whole numbers and have to be equal.  Weights: the chosen scores, their sum and the quotient in 64
bits, then one rounding to fp32: half a step, 2^-24 of the value (and half the smallest
subnormal).  Exponentials, sums and reciprocals in 64 bits are good to a few steps,
2^-48 together.  Softmax weights that are not renormalised may take the sum over all experts (added up in 64
bits) from fp32 exponentials: each is off by half a step of its argument d = l - max (relative
|d| 2^-24, as exp' = exp) and by at most two steps of its own (2^-22), so the sum is off by at most
sum e^d (|d| 2^-24 + 2^-22) / sum e^d.
"""

import math

import numpy as np

LOWEST = {"fp32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38, "fp16": -65504.0}


def _order(keys):
    """Indices by falling key, equal keys by rising index."""
    return sorted(range(len(keys)), key=lambda i: (-keys[i], i))


def route(logits, dtype, top_k, score, bias=None, n_groups=1, top_groups=1, by="max", renormalise=True, scale=1.0):
    """(ids int32 [T, k], weights fp64 [T, k], tolerances [T, k]) of logits given as fp64 values."""
    T, E = logits.shape
    per = E // n_groups
    ids = np.full((T, top_k), -1, dtype=np.int32)
    w = np.full((T, top_k), np.nan)
    tol = np.zeros((T, top_k))
    for t in range(T):
        l = [float(v) for v in logits[t]]
        b = [0.0] * E if bias is None else [float(v) for v in bias]
        by_logit = [v <= LOWEST[dtype] for v in l]
        masked = [m or c == -math.inf for m, c in zip(by_logit, b)]
        if any(not m and (math.isnan(v) or (score == "softmax" and v == math.inf) or math.isnan(c) or c == math.inf)
               for m, v, c in zip(masked, l, b)):
            continue
        if score == "sigmoid":
            # e^-l past 64 bits is infinite, and the score then zero
            with np.errstate(over="ignore"):
                s = [0.0 if m else float(1.0 / (1.0 + np.exp(-v))) for m, v in zip(by_logit, l)]
        else:
            # an expert that its bias alone masks stays in the sum, whatever its logit
            live = [v for m, v in zip(by_logit, l) if not m]
            top = max(live) if live else 0.0
            e = [0.0 if m else math.exp(v - top) for m, v in zip(by_logit, l)]
            total = math.fsum(e)
            s = [v / total if total else 0.0 for v in e]
        c = [x + y for x, y in zip(s, b)]
        order_by = l if bias is None else c
        kept = list(range(n_groups))
        if top_groups < n_groups:
            of = []
            for g in range(n_groups):
                mine = range(g * per, (g + 1) * per)
                if by == "max":
                    of.append(max([order_by[e] for e in mine if not masked[e]], default=-math.inf))
                else:
                    best = sorted((c[e] for e in mine if not masked[e]), reverse=True)[:2]
                    of.append(sum(best) if best else -math.inf)
            kept = sorted(_order(of)[:top_groups])
        pool = [e for g in kept for e in range(g * per, (g + 1) * per)]
        pool.sort(key=lambda e: (masked[e], 0.0 if masked[e] else -order_by[e], e))
        chosen = pool[:top_k]
        v = [0.0 if masked[e] else s[e] for e in chosen]
        off = 2.0 ** -48
        if renormalise:
            total = math.fsum(v)
            v = [x / total if total else 0.0 for x in v]
        elif score == "softmax":
            off += sum(x * (abs(y - top) * 2.0 ** -24 + 2.0 ** -22) for x, y, m in zip(s, l, by_logit) if not m)
        ids[t] = chosen
        w[t] = [x * scale for x in v]
        tol[t] = [x * scale * (2.0 ** -24 + off) + 2.0 ** -150 for x in v]
    return ids, w, tol
