"""The FP8 mixture-of-experts block of the examples under losses whose gradients
are not tensors in memory: a sum's is one number, expanded."""

import pytest
import torch

from tests.test_gpu_moe_block_example import load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loss", ["out", "stream", "both"])
def test_gradients_of_sums(loss):
    """As those of the same numbers in memory."""
    ex = load()
    torch.manual_seed(7)
    block = ex.MoEBlock(128, 128, 8, 2)
    x, residual = (torch.randn(65, 128, device="cuda", dtype=torch.bfloat16, requires_grad=True) for _ in range(2))
    leaves = [x, residual] + list(block.parameters())
    out, h, _ = block(x, residual)
    terms = [t for t, used in ((out, loss != "stream"), (h, loss != "out")) if used]
    got = torch.autograd.grad(sum(t.sum() for t in terms), leaves, retain_graph=True, allow_unused=True)
    want = torch.autograd.grad(terms, leaves, [torch.ones_like(t) for t in terms], allow_unused=True)
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    assert got[0] is not None and torch.isfinite(got[0]).all()
