"""Performance cases of scored routing and of 8-bit integer products.

``listed()`` and ``draw()`` give cases, ``prepare`` makes what a program has in
hand before the call, ``run`` makes one call: in plain elementary torch
operations while ``own`` is false, through ``quantized_expert_gemv_moe_amd``
while it is true.  ``exact`` gives the same outputs from the definitions in 64
bits.

Operators
  route    top-k of scored experts: softmax or sigmoid scores, a bias that only the choice
           sees, groups of experts of which the best are kept, weights renormalised
           and scaled; with the plan that the expert products take where asked for
  i8       out = residual + f(sx[r] sw[n] sum_k qx qw + bias), plain or gated, of 8-bit
           integer weights with a scale for each channel; x is quantised row by row within
           the call, or comes as integers with a scale for each row
  i8 per expert  the same product over a routed batch, every expert its own rows
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1}


# -------------------------------------------------------------------- cases
def _route(tokens, experts, top_k, score, dtype="fp32", bias=False, groups=1, keep=1, by="max", renorm=True, scale=1.0,
           plan=False, zipf=0.0):
    return dict(op="route", tokens=tokens, experts=experts, top_k=top_k, score=score, dtype=dtype, bias=bias,
                groups=groups, keep=keep, by=by, renorm=renorm, scale=scale, plan=plan, zipf=zipf)


def _dense(rows, k, n, x="bf16", out="bf16", act="none", gated=False, bias=False, residual=False, pad=0, clamp=0.0):
    """``pad``: extra elements between the rows of x and of out (0 = packed)."""
    return dict(op="dense", rows=rows, k=k, n=n, x=x, out=out, act=act, gated=gated, bias=bias, residual=residual,
                pad=pad, clamp=clamp)


def _experts(tokens, experts, top_k, k, n, x="bf16", out="bf16", act="none", gated=False, bias=False, rows="token",
             zipf=0.0, clamp=0.0):
    return dict(op="experts", tokens=tokens, experts=experts, top_k=top_k, k=k, n=n, x=x, out=out, act=act,
                gated=gated, bias=bias, rows=rows, zipf=zipf, clamp=clamp)


def listed():
    cases = [
        # one decoded token: sigmoid scores, balance bias, the best 4 of 8 groups, and its plan (latency)
        ("route_sigmoid_1", _route(1, 256, 8, "sigmoid", bias=True, groups=8, keep=4, by="top2", scale=2.5, plan=True)),
        # a ragged serving batch of a small mixture, bf16 logits, weights not renormalised
        ("route_softmax_77", _route(77, 60, 4, "softmax", dtype="bf16", renorm=False)),
        # long prompts through the grouped, biased router
        ("route_sigmoid_8192", _route(8192, 256, 8, "sigmoid", bias=True, groups=8, keep=4, by="top2", scale=2.5)),
        # long prompts through the plain router
        ("route_softmax_16384", _route(16384, 128, 8, "softmax", zipf=0.5)),
        # one decoded token through a shared expert's gate and up (latency)
        ("i8_gated_1", _dense(1, 2048, 768, act="silu", gated=True)),
        # a ragged serving batch through a biased layer of odd sizes
        ("i8_odd_77", _dense(77, 1003, 1357, x="fp16", out="fp16", act="gelu", bias=True, residual=True, pad=5)),
        # a prefill chunk through a shared expert's gate and up
        ("i8_gated_1024", _dense(1024, 2048, 768, act="silu", gated=True)),
        # a long prompt through the second half of a dense block, quantised beforehand
        ("i8_prefill_8192", _dense(8192, 8192, 4096, x="int8", bias=True, residual=True)),
        # one decoded token through its eight experts' gate and up (latency)
        ("i8_experts_1", _experts(1, 128, 8, 2048, 768, act="silu", gated=True)),
        # a decode batch of 32 with skewed expert popularity, down projections into fp32 rows
        ("i8_experts_down_32", _experts(32, 128, 8, 768, 2048, out="fp32", rows="slot", zipf=1.1)),
        # a prefill chunk: every expert holds about 64 rows
        ("i8_experts_1024", _experts(1024, 128, 8, 2048, 768, act="silu", gated=True)),
        # long prompts, about 1024 rows an expert with skewed popularity
        ("i8_experts_16384", _experts(16384, 128, 8, 2048, 768, act="silu", gated=True, zipf=0.5)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over the logarithm of the range: a multiple of 64 or of 16 in most
    draws, any number, odd ones too, in the others."""
    v = _log_int(rng, lo, hi)
    step = rng.choice([64, 64, 16, 1])
    return max(lo, min(hi, v // step * step if v >= step else v))


def draw(rng):
    op = rng.choice(["route", "dense", "experts"])
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 4, 8])
        per = _log_int(rng, 4, 256) if groups == 1 else _log_int(rng, 2, 256 // groups)
        keep = rng.randint(1, groups)
        tokens = _log_int(rng, 1, 16384)
        while tokens * per * groups > 16384 * 128:
            tokens //= 2
        return _route(tokens, per * groups, rng.randint(1, min(8, per * keep)), score,
                      dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), bias=rng.random() < 0.5, groups=groups,
                      keep=keep, by=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]), plan=tokens <= 64 and rng.random() < 0.5,
                      zipf=rng.choice([0.0, 0.5, 1.1]))
    x = rng.choice(["bf16", "bf16", "fp16", "fp32", "int8"])
    out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    act = rng.choice(["none", "silu", "gelu_tanh", "gelu", "relu"])
    gated = act in ("silu", "gelu_tanh") and rng.random() < 0.7
    if op == "dense":
        rows, k, n = _log_int(rng, 1, 8192), _size(rng, 64, 8192), _size(rng, 64, 4096)
        gated = gated and rng.random() < 0.6
        while rows > 1 and 2.0 * rows * k * n * (2 if gated else 1) > 4.0e11:
            rows //= 2
        return _dense(rows, k, n, x=x, out=out, act=act, gated=gated, bias=rng.random() < 0.5,
                      residual=rng.random() < 0.5, pad=rng.choice([0, 0, 0, 16, 64, 3]),
                      clamp=rng.choice([0.0, 0.0, 10.0]))
    experts = _log_int(rng, 2, 256)
    k, n = _size(rng, 64, 4096), _size(rng, 64, 2048)
    while experts > 2 and experts * k * n * (2 if gated else 1) > 2.0e9:
        experts //= 2
    top_k = rng.randint(1, min(8, experts))
    tokens = _log_int(rng, 1, 16384)
    while tokens > 1 and 2.0 * tokens * top_k * k * n * (2 if gated else 1) > 4.0e11:
        tokens //= 2
    return _experts(tokens, experts, top_k, k, n, x=x, out=out, act=act, gated=gated, bias=rng.random() < 0.4,
                    rows=rng.choice(["token", "slot", "sorted"]), zipf=rng.choice([0.0, 0.5, 1.1]),
                    clamp=rng.choice([0.0, 0.0, 10.0]))


# ------------------------------------------------------------------- inputs
def _logits(case, seed):
    """Normal logits with a popularity bias of -zipf ln(rank) over a random order of the experts."""
    rng = np.random.default_rng(seed)
    T, E = case["tokens"], case["experts"]
    logits = rng.standard_normal((T, E), dtype=np.float32)
    if case["zipf"]:
        logits -= (case["zipf"] * np.log(rng.permutation(E) + 1)).astype(np.float32)
    return logits


def _choice(case, seed):
    """Routing of a batch on the host for the expert products: idx [T, k] by falling logits."""
    return np.argsort(-_logits(case, seed), axis=1, kind="stable")[:, :case["top_k"]].astype(np.int32)


def _normal(gen, shape, dtype, std):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def _codes(gen, shape):
    """8-bit integers as normal values have them once the largest of a few thousand is 127."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in out.view(-1, shape[-1]).split(1 << 16):
        part.copy_(torch.empty(part.shape, device="cuda").normal_(0.0, 33.0, generator=gen).round_().clamp_(-127, 127))
    return out


def _scales(gen, shape, mean):
    return torch.empty(shape, device="cuda").uniform_(0.8 * mean, 1.2 * mean, generator=gen)


def _inputs(case, seed):
    """Everything both forms take: device tensors, and the routing's bounds on the host."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "bias": None}
    if case["op"] == "route":
        s["logits"] = torch.from_numpy(_logits(case, seed)).cuda().to(_DTYPES[case["dtype"]])
        if case["bias"]:
            s["bias"] = _normal(gen, (case["experts"],), torch.float32, 0.1)
        return s
    s |= {"residual": None, "bias_up": None, "w_up": None, "w_up_scale": None, "x_scale": None}
    K, N, odt = case["k"], case["n"], _DTYPES[case["out"]]
    if case["op"] == "dense":
        rows, x_rows, pad, lead = case["rows"], case["rows"], case["pad"], ()
    else:
        idx = _choice(case, seed)
        rows, pad, lead = idx.size, 0, (case["experts"],)
        x_rows = case["tokens"] if case["rows"] == "token" else rows
        s["idx"] = torch.from_numpy(idx).cuda()
        slots = np.argsort(idx.reshape(-1), kind="stable")
        s["bounds"] = np.searchsorted(idx.reshape(-1)[slots], np.arange(case["experts"] + 1)).tolist()
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
    if case["x"] == "int8":
        s["x"], s["x_scale"] = _codes(gen, (x_rows, K + pad))[:, :K], _scales(gen, (x_rows,), 1.0 / 33.0)
    else:
        s["x"] = _normal(gen, (x_rows, K + pad), _DTYPES[case["x"]], 1.0)[:, :K]
    s["out"] = torch.empty((rows, N + pad), dtype=odt, device="cuda")[:, :N]
    if case.get("residual"):
        s["residual"] = _normal(gen, (rows, N), odt, 1.0)
    for name in ("w", "w_up") if case["gated"] else ("w",):
        s[name] = _codes(gen, lead + (N, K))
        s[name + "_scale"] = _scales(gen, lead + (N,), 0.9 / 33.0 / math.sqrt(K))
    if case["bias"]:
        s["bias"] = _normal(gen, lead + (N,), torch.bfloat16, 0.3)
        if case["gated"]:
            s["bias_up"] = _normal(gen, lead + (N,), torch.bfloat16, 0.3)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import quantized_expert_gemv_moe_amd as moe

        s["moe"] = moe
        if case["op"] == "route":
            s["router"] = moe.Router(case["experts"], case["top_k"], score=case["score"], bias=s["bias"],
                                     n_groups=case["groups"], top_groups=case["keep"], group_score=case["by"],
                                     renormalise=case["renorm"], scale=case["scale"])
            return s
        s["linear"] = moe.LinearInt.from_tensors(s["w"], s["w_scale"], bias=s["bias"], w_up=s["w_up"],
                                                w_up_scale=s["w_up_scale"], bias_up=s["bias_up"],
                                                activation=case["act"], out_dtype=_DTYPES[case["out"]],
                                                clamp_limit=case["clamp"])
        if case["op"] == "dense":
            s["workspace"] = moe.alloc_matmul_int_workspace(s["linear"], case["rows"])
        else:
            s["plan"] = moe.expert_plan(s["idx"], case["experts"])
            s["workspace"] = moe.alloc_grouped_int_workspace(s["linear"], s["idx"].numel(), s["x"].shape[0])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        moe = state["moe"]
        if c["op"] == "route":
            if not c["plan"]:
                return moe.router_topk(state["router"], state["logits"])
            idx, w, p = moe.router_plan(state["router"], state["logits"])
            return idx, w, [p.counts, p.offsets, p.sorted_slots, p.unique_experts, p.n_unique, p.work]
        if c["op"] == "dense":
            return moe.matmul_int(state["linear"], state["x"], x_scale=state["x_scale"], residual=state["residual"],
                                 out=state["out"], workspace=state["workspace"])
        return moe.grouped_matmul_int(state["linear"], state["x"], state["plan"], c["tokens"] * c["top_k"],
                                     top_k=c["top_k"], rows=c["rows"], x_scale=state["x_scale"], out=state["out"],
                                     workspace=state["workspace"])
    if c["op"] == "route":
        return _plain_route(state)
    if c["op"] == "dense":
        return _plain_dense(state)
    return _plain_experts(state)


def _plain_route(s):
    """The order of the experts is that of numbers that may lie next to one another: 64 bits."""
    c = s["case"]
    T, E, G = c["tokens"], c["experts"], c["groups"]
    lg = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-lg))
    else:
        e = torch.exp(lg - lg.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    value = score if s["bias"] is None else score + s["bias"].double()
    order_by = lg if s["bias"] is None else value  # scores rise with their logits
    if c["keep"] < G:
        if c["by"] == "max":
            of_group = order_by.view(T, G, E // G).amax(dim=2)
        else:
            best = torch.sort(value.view(T, G, E // G), dim=2, descending=True).values
            of_group = best[:, :, :2].sum(dim=2)
        kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        out = torch.ones((T, G), dtype=torch.bool, device=lg.device).scatter_(1, kept, False)
        order_by = order_by.masked_fill(out[:, :, None].expand(T, G, E // G).reshape(T, E), -math.inf)
    idx = torch.sort(order_by, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    idx, w = idx.to(torch.int32), (w * c["scale"]).float()
    return (idx, w, _plain_plan(idx, E)) if c["plan"] else (idx, w)


def _plain_plan(idx, E):
    flat = idx.reshape(-1).long()
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(dim=0)
    ends = torch.cumsum(counts, dim=0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    slots = torch.sort(flat, stable=True).indices
    used = counts > 0
    ids = torch.sort((~used).to(torch.int32), stable=True).indices  # the experts in use, ascending, first
    there = used[ids]
    first = slots[offsets[:-1].clamp(max=flat.numel() - 1)]
    work = torch.stack([ids, offsets[:-1][ids], counts[ids], first[ids]], dim=1)
    end = torch.tensor([-1, flat.numel(), 0, 0], device=flat.device)
    return [t.to(torch.int32) for t in (counts, offsets, slots, torch.where(there, ids, -1), used.sum().reshape(1),
                                        torch.where(there[:, None], work, end))]


def _plain_act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        # 0.5 (1 + tanh a) = 1 / (1 + exp(-2 a)), without the cancellation at negative a
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    return z


def _plain_quantise(x, scale):
    """Integers and scales of the rows; 64 bits, as quotients half way between two integers go to the even one."""
    if scale is not None:
        return x.float(), scale
    x = x.float()
    top = x.abs().amax(dim=1)
    # a row of zeros has zeros for codes
    per = torch.where(top > 0, top, torch.ones_like(top)).double()
    return torch.round(x.double() * 127.0 / per[:, None]).float(), top / 127.0


def _plain_product(c, q, scale, w, w_scale, w_up, w_up_scale, bias, bias_up):
    # integers below 2^24: their sums are exact in fp32 in any order
    z = (q @ w.float().t()) * scale[:, None] * w_scale
    if bias is not None:
        z = z + bias.float()
    if c["clamp"]:
        z = z.clamp(-c["clamp"], c["clamp"])
    z = _plain_act(z, c["act"])
    if c["gated"]:
        u = (q @ w_up.float().t()) * scale[:, None] * w_up_scale
        if bias_up is not None:
            u = u + bias_up.float()
        if c["clamp"]:
            u = u.clamp(-c["clamp"], c["clamp"])
        z = z * u
    return z


def _plain_dense(s):
    q, scale = _plain_quantise(s["x"], s["x_scale"])
    z = _plain_product(s["case"], q, scale, s["w"], s["w_scale"], s["w_up"], s["w_up_scale"], s["bias"], s["bias_up"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    s["out"].copy_(z)
    return s["out"]


def _plain_experts(s):
    """A loop over the experts in use: they differ in their rows, and a stack of all
    of them, padded to the largest, would be mostly padding."""
    c = s["case"]
    q, scale = _plain_quantise(s["x"], s["x_scale"])

    def of(name, e):
        return None if s[name] is None else s[name][e]

    for e in range(c["experts"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo == hi:
            continue
        slots = s["slots"][lo:hi]
        at = slice(lo, hi) if c["rows"] == "sorted" else slots // c["top_k"] if c["rows"] == "token" else slots
        z = _plain_product(c, q[at], scale[at], s["w"][e], s["w_scale"][e], of("w_up", e), of("w_up_scale", e),
                           of("bias", e), of("bias_up", e))
        s["out"][at if c["rows"] == "sorted" else slots] = z.to(s["out"].dtype)
    return s["out"]


# ------------------------------------------------------------- definitions
def _before(v):
    """For every number of the last axis, how many stand before it: the greater ones, and equal ones further left."""
    n = v.shape[-1]
    left = torch.ones((n, n), dtype=torch.bool, device=v.device).tril(-1)  # [i, j]: j left of i
    mine, other = v[..., :, None], v[..., None, :]
    return ((other > mine) | ((other == mine) & left)).sum(dim=-1)


def _exact_route(case, s):
    E, G, k = case["experts"], case["groups"], case["top_k"]
    per = E // G
    ids, weights = [], []
    for part in s["logits"].split(max(1, (1 << 26) // (E * E))):
        v = part.double()
        if case["score"] == "sigmoid":
            p = torch.sigmoid(v)
        else:
            p = torch.exp(v - torch.logsumexp(v, dim=1, keepdim=True))
        value = p if s["bias"] is None else p + s["bias"].double()
        by = v if s["bias"] is None else value
        if case["keep"] < G:
            if case["by"] == "max":
                g = by.reshape(-1, G, per).max(dim=2).values
            else:
                g = torch.topk(value.reshape(-1, G, per), min(2, per), dim=2).values.sum(dim=2)
            live = (_before(g) < case["keep"]).repeat_interleave(per, dim=1)
            by = torch.where(live, by, torch.full_like(by, -math.inf))
        place = _before(by)
        mine = torch.nonzero(place < k)  # row by row, ascending experts
        idx = torch.empty((v.shape[0], k), dtype=torch.long, device=v.device)
        idx[mine[:, 0], place[mine[:, 0], mine[:, 1]]] = mine[:, 1]
        w = torch.take_along_dim(p, idx, dim=1)
        if case["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        ids.append(idx)
        weights.append(w * case["scale"])
    idx = torch.cat(ids)
    out = [idx.to(torch.int32), torch.cat(weights)]
    if case["plan"]:
        flat = idx.reshape(-1).tolist()
        lists = [[i for i, e in enumerate(flat) if e == want] for want in range(E)]
        offsets = np.cumsum([0] + [len(m) for m in lists]).tolist()
        used = [e for e in range(E) if lists[e]]
        work = [[e, offsets[e], len(lists[e]), lists[e][0]] for e in used] + [[-1, len(flat), 0, 0]] * (E - len(used))
        out.append([torch.tensor(t, dtype=torch.int32) for t in (
            [len(m) for m in lists], offsets, sum(lists, []), used + [-1] * (E - len(used)), [len(used)], work)])
    return tuple(out)


def _f64(act, v):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":  # 0.5 (1 + tanh a) = sigmoid(2 a)
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "relu":
        return torch.relu(v)
    return v


def _affine64(x, w, w_scale, b, limit):
    v = torch.matmul(x, (w.double() * w_scale.double()[:, None]).transpose(0, 1))
    if b is not None:
        v += b.double()
    return torch.clip(v, -limit, limit) if limit else v


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, None]
    else:  # the values that the codes stand for
        top = x.abs().max(dim=1, keepdim=True).values
        x = torch.where(top > 0, torch.round(x * 127.0 / top) * top / 127.0, x)

    def product(rows, pick):
        v = _f64(case["act"], _affine64(rows, pick("w"), pick("w_scale"), pick("bias"), case["clamp"]))
        if case["gated"]:
            v *= _affine64(rows, pick("w_up"), pick("w_up_scale"), pick("bias_up"), case["clamp"])
        return v

    if case["op"] == "dense":
        v = product(x, s.get)
        return v if s["residual"] is None else v + s["residual"].double()
    flat = s["idx"].reshape(-1)
    out = torch.zeros((flat.numel(), case["n"]), dtype=torch.float64, device="cuda")
    first = 0
    for e in range(case["experts"]):
        mine = torch.nonzero(flat == e).reshape(-1)  # this expert's slots, ascending
        here = torch.arange(first, first + mine.numel(), device="cuda")  # their sorted places
        first += mine.numel()
        if mine.numel() == 0:
            continue
        at = here if case["rows"] == "sorted" else mine
        of = mine.div(case["top_k"], rounding_mode="floor") if case["rows"] == "token" else at
        out[at] = product(x.index_select(0, of), lambda n: None if s[n] is None else s[n][e])
    return out


def work(case):
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        plan = (E * 7 + 2 + T * k) * 4 if case["plan"] else 0
        return {"bytes": T * E * _BYTES[case["dtype"]] + T * k * 8 + (E * 4 if case["bias"] else 0) + plan,
                "flops": T * E * 8}
    n, k_in, os_ = case["n"], case["k"], _BYTES[case["out"]]
    mats = 2 if case["gated"] else 1
    if case["op"] == "dense":
        rows = x_rows = case["rows"]
        groups, extra = 1, rows * n * os_ if case["residual"] else 0
    else:
        rows = case["tokens"] * case["top_k"]
        groups = len(np.unique(_choice(case, 0)))  # distinct experts of one such batch
        x_rows = case["tokens"] if case["rows"] == "token" else rows
        extra = rows * 4
    if case["bias"]:
        extra += groups * mats * n * 2
    if case["x"] == "int8":
        extra += x_rows * 4
    return {"bytes": x_rows * k_in * _BYTES[case["x"]] + groups * mats * n * (k_in + 4) + rows * n * os_ + extra,
            "flops": 2 * rows * n * k_in * mats}
