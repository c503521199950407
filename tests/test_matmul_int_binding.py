"""Refusals of the integer products' wrappers that need no GPU."""

import pytest
import torch

import quantized_expert_gemv_moe_amd as moe


def test_weights_need_their_scales():
    w = torch.zeros((4, 16), dtype=torch.int8)
    with pytest.raises(ValueError, match="w_scale"):
        moe.LinearInt.from_tensors(w, None)
