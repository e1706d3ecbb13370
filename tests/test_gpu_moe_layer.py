"""The FP8 mixture-of-experts layer of the examples against the same layer in
fp32 on the projected weights.

An E4M3 value with its block's scale is off by at most 2^-4 of itself, and by
2^-4 / sqrt(3) = 0.036 in the mean square.  The weights are exact.  At most
three such roundings lie between an input and an output of the layer or of
its backward pass (the input of each layer, and the gradient), so that
independent errors add up to 0.036 * sqrt(3) = 0.0625; the bound is twice that."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = 0.125


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_moe_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_moe_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,experts,topk,width,hidden", [(300, 4, 2, 256, 384), (1, 8, 1, 128, 128), (65, 16, 4, 640, 256)])
def test_layer_and_gradients(tokens, experts, topk, width, hidden):
    ex = load()
    torch.manual_seed(tokens)
    layer = ex.MoELayer(width, hidden, experts, topk)
    x = torch.randn(tokens, width, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    off = ex.compare(layer, x)
    # with topk 1 the weights are one whatever the router says: its gradient is nothing but rounding
    bad = {k: v for k, v in off.items() if not v <= BOUND and not (k == "router" and topk == 1)}
    assert not bad, off
