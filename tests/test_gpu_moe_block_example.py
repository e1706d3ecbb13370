"""The FP8 mixture-of-experts block of the examples against the same block in
fp32 on the projected weights.

An E4M3 value with its block's scale is off by at most 2^-4 of itself, and by
2^-4 / sqrt(3) = 0.036 in the mean square.  The weights are exact.  At most six
such roundings lie between an input and a gradient of a weight (the norm's
output, as it enters both factors of the activation, the two gradients that
enter products, and the two operands of the weight's gradient): independent
errors add up to 0.036 * sqrt(6) = 0.088; the bound is twice that.  What is
not quantized on its way (the residual stream) is rounded to bf16 once."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = 0.176


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_moe_block.py")
    spec = importlib.util.spec_from_file_location("fp8_moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,experts,topk,width,hidden,groups,topk_groups", [(300, 8, 2, 256, 384, 1, 1), (1, 8, 2, 128, 128, 4, 2), (65, 16, 4, 640, 256, 4, 2)])
def test_block_and_gradients(tokens, experts, topk, width, hidden, groups, topk_groups):
    ex = load()
    torch.manual_seed(tokens)
    block = ex.MoEBlock(width, hidden, experts, topk, groups, topk_groups)
    x, residual = (torch.randn(tokens, width, device="cuda", dtype=torch.bfloat16, requires_grad=True) for _ in range(2))
    off = ex.compare(block, x, residual)
    bad = {k: v for k, v in off.items() if not v <= (2.0**-8 if "stream" in k else BOUND)}
    assert not bad, off
