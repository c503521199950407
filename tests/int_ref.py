"""The 8-bit integer products and the quantisation of rows in 64 bits, and how far the kernels
may be from them.

Codes are whole numbers and have to be equal: 127 x / m is divided in fp64, where 127 x is exact
(31 bits), a quotient half way between two integers is exact, and any other is at least 2^-32 of itself away
from the middle, so that the rounding to an integer is the exact quotient's.  The scale m / 127 is one
fp32 division.

A product's integer sum S is exact.  z = fp32(S) * fp32(sx sw): three roundings, at most
(1 + u)^3 - 1 < 3.001 u of |z| with u = 2^-24; a bias adds u (|z| + |b|).  From there f, gate,
residual and the store as matmul_ref has them."""

import torch

from matmul_ref import U, _fn, check, half_step  # noqa: F401


def quantize(x):
    """(codes fp64, scales fp32) of rows on any device."""
    x = x.float()
    m = x.abs().amax(dim=1)
    m = torch.where(torch.isnan(x).any(dim=1), torch.full_like(m, float("nan")), m)
    fine = torch.isfinite(m)
    per = torch.where(fine & (m > 0), m, torch.ones_like(m)).double()
    q = torch.round(torch.where(fine[:, None], x, torch.zeros_like(x)).double() * 127.0 / per[:, None])
    scale = (m.cpu() / 127.0).to(x.device)  # one correctly rounded division
    return q, torch.where(fine, scale, torch.full_like(scale, float("nan")))


def _affine(q, sx, w, sw, b, clamp):
    z = (q @ w.double().t()) * sx.double()[:, None] * sw.double()[None, :]
    err = 3.001 * U * z.abs() + 2.0 ** -149
    if b is not None:
        err = err + 1.001 * U * (z.abs() + b.double().abs())
        z = z + b.double()
    if clamp:
        z = torch.where(z > clamp, torch.full_like(z, clamp), torch.where(z < -clamp, torch.full_like(z, -clamp), z))
    return z, err


def product(q, sx, w, sw, bias=None, w_up=None, sw_up=None, bias_up=None, act="none", clamp=0.0, residual=None,
            out_dtype=torch.float32):
    """(value, tolerance), both fp64; q the codes as fp64, their sums exact there."""
    z, ez = _affine(q, sx, w, sw, bias, clamp)
    f, slope, arg = _fn(z, act)
    err = slope * ez + (16 + 4 * arg) * U * f.abs()
    if w_up is not None:
        u, eu = _affine(q, sx, w_up, sw_up, bias_up, clamp)
        err = err * (u.abs() + eu) + f.abs() * eu + 2 * U * (f * u).abs()
        f = f * u
    if residual is not None:
        f = f + residual.double()
        err = err + U * f.abs()
    return f, err + half_step(out_dtype, f.abs() + err)
