"""Where a column stands changes no bit of it: the last columns of the large tiles of the integer products
are computed by two workgroups at different places of their tiles, which both write them."""

import pytest
import torch

import quantized_expert_gemv_moe_amd as moe
from gpu_helpers import log
from test_gpu_matmul_int import BF16, F16, F32, I8, gen, make_x, normal

pytestmark = pytest.mark.gpu


def linear(g, N, K, gated, bias, act, out, clamp, by):
    """The same columns, `by` places further round; made from g alone."""
    def codes():
        return torch.empty((N, K), device="cuda").normal_(0.0, 33.0, generator=g).round_().clamp_(-127, 127).to(I8)

    def scales():
        return torch.empty(N, device="cuda").uniform_(0.5, 1.5, generator=g) / (33.0 * K ** 0.5)

    t = {"w": codes(), "w_scale": scales()}
    if gated:
        t |= {"w_up": codes(), "w_up_scale": scales()}
    for name in ("bias", "bias_up")[:0 if bias is None else 1 + gated]:
        t[name] = normal(g, (N,), bias)
    t = {k: v.roll(by, 0).contiguous() for k, v in t.items()}
    return moe.LinearInt.from_tensors(activation=act, out_dtype=out, clamp_limit=clamp, **t)


# rows, K, N: the 256 x 256 and the 128 x 128 tile (tests of the choice of kernel have the same sizes), last tiles of a few
# columns, of all but a few, of an odd number, and of a half
@pytest.mark.parametrize("gated,rows,K,N", [(False, 5986, 1088, 2056), (False, 5986, 1088, 2094), (False, 5986, 1088, 2303),
                                            (False, 4486, 176, 876), (False, 4486, 176, 769), (True, 3918, 518, 1859),
                                            (True, 3918, 518, 1798), (True, 2210, 38, 1577)])
@pytest.mark.parametrize("out", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
def test_a_column_is_the_same_wherever_it_stands(gated, rows, K, N, out):
    g = gen(N)
    x, xs, _, _ = make_x(g, rows, K, I8)
    residual = normal(g, (rows, N), out)
    other = normal(g, (rows, N), F16 if out is BF16 else BF16)
    for act in ("none", "silu", "gelu", "gelu_tanh", "relu"):
        for bias, res, clamp in ((None, None, 0.0), (BF16, residual, 0.0), (F32, None, 1.0), (None, residual, 0.0),
                                 (F16, other, 0.0)):
            log(f"[case] place gated={gated} {rows} {K} {N} {out} {act} bias={bias} residual={res is not None}")
            want = None
            for by in (0, 5, 64, N - 17):
                lin = linear(gen(N + 1), N, K, gated, bias, act, out, clamp, by)
                got = moe.matmul_int(lin, x, x_scale=xs, residual=None if res is None else res.roll(by, 1).contiguous())
                got = got.roll(-by, 1)
                torch.cuda.synchronize()
                want = got if want is None else want
                bits = torch.int32 if out is F32 else torch.int16
                off = got.contiguous().view(bits) != want.contiguous().view(bits)
                assert not bool(off.any()), f"{act} by={by}: {int(off.sum())} values, columns {off.any(0).nonzero()[:8].flatten().tolist()}"
