"""Performance cases of the dense, grouped and combining operators.

``listed()`` and ``draw()`` give cases, ``prepare`` makes what a program has in
hand before the call, ``run`` makes one call: in plain elementary torch
operations (32 bits, one rounding at the end) while ``own`` is false, through
``quantized_expert_gemv_moe_amd`` while it is true.  ``exact`` gives the same
outputs from the definitions in 64 bits.

Operators
  matmul   out = residual + f(x W^T + bias), f an activation, plain or gated:
           the shared expert and the dense projections beside routed experts
  grouped  the same product per expert over a routed batch, every expert with
           its own number of rows
  combine  out[t] = residual[t] + sum_j w[t][j] y[t * k + j]
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# -------------------------------------------------------------------- cases
def _matmul(rows, k, n, dtype="bf16", out="", act="none", gated=False, bias=False, residual=False, pad=0,
            clamp=0.0):
    """``pad``: extra elements between the rows of x and of out (0 = packed)."""
    return dict(op="matmul", rows=rows, k=k, n=n, dtype=dtype, out=out or dtype, act=act, gated=gated, bias=bias,
                residual=residual, pad=pad, clamp=clamp)


def _grouped(tokens, experts, top_k, k, n, dtype="bf16", out="", act="none", gated=False, bias=False, rows="token",
             zipf=0.0, clamp=0.0):
    return dict(op="grouped", tokens=tokens, experts=experts, top_k=top_k, k=k, n=n, dtype=dtype, out=out or dtype,
                act=act, gated=gated, bias=bias, rows=rows, zipf=zipf, clamp=clamp)


def _combine(tokens, experts, top_k, n, dtype="fp32", out="bf16", residual=True):
    return dict(op="combine", tokens=tokens, experts=experts, top_k=top_k, n=n, dtype=dtype, out=out,
                residual=residual)


def listed():
    cases = [
        # one decoded token through a shared expert's gate and up (latency)
        ("matmul_gated_1", _matmul(1, 2048, 768, act="silu", gated=True)),
        # a ragged serving batch through a biased layer of odd sizes, rows that start at any 2 bytes
        ("matmul_odd_fp16_77", _matmul(77, 1003, 1357, dtype="fp16", act="gelu", bias=True, residual=True, pad=5)),
        # a small fp32 network's layer
        ("matmul_fp32_300", _matmul(300, 256, 500, dtype="fp32", act="gelu_tanh", bias=True)),
        # a prefill chunk through a shared expert's gate and up
        ("matmul_gated_1024", _matmul(1024, 2048, 768, act="silu", gated=True)),
        # a long prompt through the second half of a dense block: bias and residual
        ("matmul_prefill_8192", _matmul(8192, 8192, 4096, bias=True, residual=True)),
        # one decoded token through its eight experts' gate and up (latency)
        ("grouped_gated_1", _grouped(1, 128, 8, 2048, 768, act="silu", gated=True)),
        # a decode batch of 32 with skewed expert popularity, down projections into fp32 rows
        ("grouped_down_32", _grouped(32, 128, 8, 768, 2048, out="fp32", rows="slot", zipf=1.1)),
        # a prefill chunk: every expert holds about 64 rows
        ("grouped_gated_1024", _grouped(1024, 128, 8, 2048, 768, act="silu", gated=True)),
        # the wide clamped layer, about 96 rows an expert, 8.6 GB of weights
        ("grouped_wide_4096", _grouped(4096, 256, 6, 4096, 2048, act="silu", gated=True, clamp=10.0)),
        # long prompts, about 1024 rows an expert with skewed popularity
        ("grouped_gated_16384", _grouped(16384, 128, 8, 2048, 768, act="silu", gated=True, zipf=0.5)),
        # the end of a decode step of 8 tokens (latency)
        ("combine_8", _combine(8, 128, 8, 2048)),
        # the end of a prefill chunk's step
        ("combine_4096", _combine(4096, 256, 6, 4096)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over the logarithm of the range: a multiple of 64 or of 8 in most
    draws, any number, odd ones too, in the others."""
    v = _log_int(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(lo, min(hi, v // step * step if v >= step else v))


def draw(rng):
    op = rng.choice(["matmul", "grouped", "matmul", "grouped", "combine"])
    if op == "combine":
        experts = _log_int(rng, 8, 256)
        return _combine(_log_int(rng, 1, 4096), experts, rng.randint(1, 8), _size(rng, 64, 4096),
                        dtype=rng.choice(["fp32", "fp32", "bf16"]), out=rng.choice(["bf16", "fp16", "fp32"]),
                        residual=rng.random() < 0.7)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    act = rng.choice(["none", "silu", "gelu_tanh", "gelu", "relu"])
    gated = act in ("silu", "gelu_tanh") and rng.random() < 0.7
    out = "fp32" if rng.random() < 0.25 else dtype
    if op == "matmul":
        rows, k, n = _log_int(rng, 1, 8192), _size(rng, 64, 8192), _size(rng, 64, 4096)
        gated = gated and rng.random() < 0.6
        while rows > 1 and 2.0 * rows * k * n * (2 if gated else 1) > 4.0e11:
            rows //= 2
        return _matmul(rows, k, n, dtype=dtype, out=out, act=act, gated=gated, bias=rng.random() < 0.5,
                       residual=rng.random() < 0.5, pad=rng.choice([0, 0, 0, 8, 64, 3]),
                       clamp=rng.choice([0.0, 0.0, 10.0]))
    experts = _log_int(rng, 2, 256)
    top_k = rng.randint(1, min(8, experts))
    k, n = _size(rng, 64, 4096), _size(rng, 64, 2048)
    # at most the largest listed case's weights and its products
    while experts > 2 and experts * k * n * (2 if gated else 1) * _BYTES[dtype] > 4.0e9:
        experts //= 2
    top_k = min(top_k, experts)
    tokens = _log_int(rng, 1, 16384)
    while tokens > 1 and 2.0 * tokens * top_k * k * n * (2 if gated else 1) > 4.0e11:
        tokens //= 2
    return _grouped(tokens, experts, top_k, k, n, dtype=dtype, out=out, act=act, gated=gated,
                    bias=rng.random() < 0.4, rows=rng.choice(["token", "slot", "sorted"]),
                    zipf=rng.choice([0.0, 0.5, 1.1]), clamp=rng.choice([0.0, 0.0, 10.0]))


# ------------------------------------------------------------------- inputs
def _route(case, seed):
    """Seeded routing of a batch on the host: idx [T, k] in falling order of the logits
    (normal, with a popularity bias of -zipf * ln(rank) over a random order of the
    experts), and the softmax of the kept logits."""
    rng = np.random.default_rng(seed)
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    logits = rng.standard_normal((T, E), dtype=np.float32)
    if case.get("zipf"):
        rank = rng.permutation(E) + 1
        logits -= (case["zipf"] * np.log(rank)).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    kept = np.take_along_axis(logits, idx.astype(np.int64), axis=1)
    p = np.exp(kept - kept[:, :1])
    return idx, (p / p.sum(axis=1, keepdims=True)).astype(np.float32)


def _normal(gen, shape, dtype, std):
    if len(shape) == 3:  # stacked experts: one at a time, so no fp32 copy of the whole stack
        out = torch.empty(shape, dtype=dtype, device="cuda")
        for e in range(shape[0]):
            out[e] = torch.empty(shape[1:], dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
        return out
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def _inputs(case, seed):
    """Everything both forms take: device tensors, and the routing's bounds on the host."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "residual": None, "bias": None, "bias_up": None, "w_up": None}
    dt, odt = _DTYPES[case["dtype"]], _DTYPES[case["out"]]
    n = case["n"]
    if case["op"] != "matmul":
        idx, w = _route(case, seed)
        E, k = case["experts"], case["top_k"]
        s["idx"], s["topk_w"] = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()
        slots = np.argsort(idx.reshape(-1), kind="stable")
        s["bounds"] = np.searchsorted(idx.reshape(-1)[slots], np.arange(E + 1)).tolist()
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
        n_slots = idx.size
    if case["op"] == "combine":
        s["y"] = _normal(gen, (n_slots, n), dt, 0.5)
        if case["residual"]:
            s["residual"] = _normal(gen, (case["tokens"], n), odt, 1.0)
        s["out"] = torch.empty((case["tokens"], n), dtype=odt, device="cuda")
        return s
    k_in = case["k"]
    std = 0.9 / math.sqrt(k_in)
    if case["op"] == "matmul":
        rows, pad = case["rows"], case["pad"]
        s["x"] = _normal(gen, (rows, k_in + pad), dt, 1.0)[:, :k_in]
        s["out"] = torch.empty((rows, n + pad), dtype=odt, device="cuda")[:, :n]
        if case["residual"]:
            s["residual"] = _normal(gen, (rows, n), odt, 1.0)
        lead = ()
    else:
        s["x"] = _normal(gen, (case["tokens"] if case["rows"] == "token" else n_slots, k_in), dt, 1.0)
        s["out"] = torch.empty((n_slots, n), dtype=odt, device="cuda")
        lead = (case["experts"],)
    s["w"] = _normal(gen, lead + (n, k_in), dt, std)
    if case["gated"]:
        s["w_up"] = _normal(gen, lead + (n, k_in), dt, std)
    if case["bias"]:
        s["bias"] = _normal(gen, lead + (n,), dt, 0.3)
        if case["gated"]:
            s["bias_up"] = _normal(gen, lead + (n,), dt, 0.3)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import quantized_expert_gemv_moe_amd as moe

        s["moe"] = moe
        if case["op"] == "grouped":
            s["plan"] = moe.expert_plan(s["idx"], case["experts"])
        if case["op"] != "combine":
            s["linear"] = moe.Linear.from_tensors(s["w"], bias=s["bias"], w_up=s["w_up"], bias_up=s["bias_up"],
                                                  activation=case["act"], out_dtype=_DTYPES[case["out"]],
                                                  clamp_limit=case["clamp"])
        if case["op"] == "matmul":
            s["workspace"] = moe.alloc_matmul_workspace(s["linear"], case["rows"])
        elif case["op"] == "grouped":
            s["workspace"] = moe.alloc_grouped_workspace(s["linear"], s["idx"].numel())
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        moe, c = state["moe"], state["case"]
        if op == "matmul":
            return moe.matmul(state["linear"], state["x"], residual=state["residual"], out=state["out"],
                              workspace=state["workspace"])
        if op == "grouped":
            return moe.grouped_matmul(state["linear"], state["x"], state["plan"], c["tokens"] * c["top_k"],
                                      top_k=c["top_k"], rows=c["rows"], out=state["out"],
                                      workspace=state["workspace"])
        return moe.combine(state["y"], state["idx"], state["topk_w"], c["experts"], residual=state["residual"],
                           out=state["out"])
    if op == "matmul":
        return _plain_matmul(state)
    if op == "grouped":
        return _plain_grouped(state)
    return _plain_combine(state)


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


def _plain_product(c, x, w, w_up, bias, bias_up):
    x = x.float()
    z = x @ w.float().t()
    if bias is not None:
        z = z + bias.float()
    if c["clamp"]:
        z = z.clamp(-c["clamp"], c["clamp"])
    z = _plain_act(z, c["act"])
    if c["gated"]:
        u = x @ w_up.float().t()
        if bias_up is not None:
            u = u + bias_up.float()
        if c["clamp"]:
            u = u.clamp(-c["clamp"], c["clamp"])
        z = z * u
    return z


def _plain_matmul(s):
    z = _plain_product(s["case"], s["x"], s["w"], s["w_up"], s["bias"], s["bias_up"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    s["out"].copy_(z)
    return s["out"]


def _plain_grouped(s):
    c = s["case"]
    for e in range(c["experts"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo == hi:
            continue
        slots = s["slots"][lo:hi]
        if c["rows"] == "sorted":
            x = s["x"][lo:hi]
        else:
            x = s["x"][slots // c["top_k"] if c["rows"] == "token" else slots]
        z = _plain_product(c, x, s["w"][e], s["w_up"][e] if c["gated"] else None,
                           s["bias"][e] if c["bias"] else None,
                           s["bias_up"][e] if c["bias"] and c["gated"] else None)
        if c["rows"] == "sorted":
            s["out"][lo:hi] = z.to(s["out"].dtype)
        else:
            s["out"][slots] = z.to(s["out"].dtype)
    return s["out"]


def _plain_combine(s):
    c = s["case"]
    y = s["y"].view(c["tokens"], c["top_k"], c["n"]).float()
    z = (y * s["topk_w"][:, :, None]).sum(dim=1)
    if s["residual"] is not None:
        z = z + s["residual"].float()
    s["out"].copy_(z)
    return s["out"]


# ------------------------------------------------------------- definitions
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


def _affine64(x, w, b, limit):
    v = torch.matmul(x, w.double().transpose(0, 1))
    if b is not None:
        v += b.double()
    return torch.clip(v, -limit, limit) if limit else v


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "combine":
        acc = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device="cuda")
        if case["residual"]:
            acc += s["residual"].double()
        rows = torch.arange(case["tokens"], device="cuda") * case["top_k"]
        for j in range(case["top_k"]):
            acc += s["topk_w"][:, j].double()[:, None] * s["y"][rows + j].double()
        return acc
    if case["op"] == "matmul":
        x = s["x"].double()
        v = _f64(case["act"], _affine64(x, s["w"], s["bias"], case["clamp"]))
        if case["gated"]:
            v *= _affine64(x, s["w_up"], s["bias_up"], case["clamp"])
        if case["residual"]:
            v += s["residual"].double()
        return v
    flat = s["idx"].reshape(-1)
    out = torch.zeros((flat.numel(), case["n"]), dtype=torch.float64, device="cuda")
    first = 0
    for e in range(case["experts"]):
        mine = torch.nonzero(flat == e).reshape(-1)  # this expert's slots, ascending
        here = torch.arange(first, first + mine.numel(), device="cuda")  # their sorted places
        first += mine.numel()
        if mine.numel() == 0:
            continue
        if case["rows"] == "token":
            x = s["x"].index_select(0, mine.div(case["top_k"], rounding_mode="floor"))
        else:
            x = s["x"].index_select(0, here if case["rows"] == "sorted" else mine)
        x = x.double()
        v = _f64(case["act"], _affine64(x, s["w"][e], s["bias"][e] if case["bias"] else None, case["clamp"]))
        if case["gated"]:
            v *= _affine64(x, s["w_up"][e], s["bias_up"][e] if case["bias"] else None, case["clamp"])
        out[here if case["rows"] == "sorted" else mine] = v
    return out


def work(case):
    es, os_ = _BYTES[case["dtype"]], _BYTES[case["out"]]
    n = case["n"]
    if case["op"] == "combine":
        T, k = case["tokens"], case["top_k"]
        return {"bytes": T * k * n * es + T * n * os_ * (2 if case["residual"] else 1) + T * k * 8,
                "flops": 2 * T * k * n}
    mats = 2 if case["gated"] else 1
    k_in = case["k"]
    if case["op"] == "matmul":
        rows, groups, x_rows = case["rows"], 1, case["rows"]
        extra = rows * n * os_ if case["residual"] else 0
    else:
        rows = case["tokens"] * case["top_k"]
        groups = len(np.unique(_route(case, 0)[0]))  # distinct experts of one such batch
        x_rows = case["tokens"] if case["rows"] == "token" else rows
        extra = rows * 4
    if case["bias"]:
        extra += groups * mats * n * es
    return {"bytes": (x_rows * k_in + groups * mats * n * k_in) * es + rows * n * os_ + extra,
            "flops": 2 * rows * n * k_in * mats}
