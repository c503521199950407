"""The unquantised products and the combine in 64 bits, and how far an fp32
evaluation with one final rounding may be from them.

Error of a sum of K fp32 products against the exact one: each of the K
additions is off by at most u = 2^-24 of the running sum, which is at most
S = sum |x||w|; as independent errors they add up to about sqrt(K) u S, and the
bound taken is (2 sqrt(K) + 16) u S (the worst case, K u S, would let a lost
element pass).  The products of bf16 and fp16 values are exact; fp32 products round once
more each, which the factor 2 covers.  Through f and the gate the error grows by |f'| <=
1.13 and by the other factor.  f itself is evaluated with a few roundings and an
exponential whose relative error is that of its argument, |a| u times a small
factor: (16 + 4 |a|) u |f|.  The store rounds once more: half a step of the
output type, eps / 2 relative (and half the smallest subnormal).
"""

import math

import torch

U = 2.0 ** -24


def half_step(dtype, ref):
    fi = torch.finfo(dtype)
    return (fi.eps / 2) * ref.abs() + fi.tiny * fi.eps / 2


def _fn(z, name):
    """f(z), |f'| bound, magnitude of the exponential's argument."""
    if name == "none":
        return z, 1.0, torch.zeros_like(z)
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z), 1.0, torch.zeros_like(z)
    if name == "silu":
        return z * torch.sigmoid(z), 1.13, z.abs()
    if name == "gelu":
        return z * torch.special.ndtr(z), 1.13, z * z / 2
    a = 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.sigmoid(a), 1.13, a.abs()


def _affine(x, w, b, clamp):
    x, w = x.double(), w.double()
    z = x @ w.t()
    s = x.abs() @ w.abs().t()
    err = (2 * math.sqrt(x.shape[1]) + 16) * U * s
    if b is not None:
        z = z + b.double()
        err = err + 2 * U * (s + b.double().abs())
    if clamp:
        z = torch.where(z > clamp, torch.full_like(z, clamp), torch.where(z < -clamp, torch.full_like(z, -clamp), z))
    return z, err


def product(x, w, bias=None, w_up=None, bias_up=None, act="none", clamp=0.0, residual=None, out_dtype=torch.float32):
    """(value, tolerance), both fp64, of f(x w^T + bias) [* (x w_up^T + bias_up)] + residual."""
    z, ez = _affine(x, w, bias, clamp)
    f, slope, arg = _fn(z, act)
    err = slope * ez + (16 + 4 * arg) * U * f.abs()
    if w_up is not None:
        u, eu = _affine(x, w_up, bias_up, clamp)
        err = err * (u.abs() + eu) + f.abs() * eu + 2 * U * (f * u).abs()
        f = f * u
    if residual is not None:
        r = residual.double()
        f = f + r
        err = err + U * f.abs()
    return f, err + half_step(out_dtype, f.abs() + err)


def combine(y, idx, w, n_experts, residual=None, out_dtype=torch.float32):
    B, k = idx.shape
    yd = y.double().view(B, k, -1) * w.double()[:, :, None]
    v = yd.sum(dim=1)
    err = (k + 2) * U * yd.abs().sum(dim=1)
    if residual is not None:
        v = v + residual.double()
        err = err + U * v.abs()
    bad = ((idx < 0) | (idx >= n_experts)).any(dim=1)
    v = torch.where(bad[:, None], torch.full_like(v, float("nan")), v)
    return v, err + half_step(out_dtype, v.abs() + err)


def check(got, want, tol, tag):
    """NaN where the definition has NaN, infinities equal, everything else within tol."""
    g, w, t = got.double().cpu(), want.double().cpu(), tol.double().cpu()
    nan = torch.isnan(w)
    assert torch.equal(torch.isnan(g), nan), f"{tag}: NaN in other places ({int(torch.isnan(g).sum())} for {int(nan.sum())})"
    big = torch.finfo(got.dtype).max
    over = (w.abs() > big) & ~nan  # beyond the type: infinity, or its largest value within half a step
    live = ~nan & ~over
    assert bool((g[over] * torch.sign(w[over]) >= big).all()), f"{tag}: wrong overflow"
    bad = live & ~((g - w).abs() <= t)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{tag}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{g.reshape(-1)[i]} for {w.reshape(-1)[i]}, tolerance {t.reshape(-1)[i]}")
