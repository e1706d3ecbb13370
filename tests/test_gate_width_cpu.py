"""Widths that two halves take out of 64 bits are refused before any launch."""

import pytest

import block_scaled_precision_x32_gb300 as mxq

INVALID, FAKE = 1, 0x10000000  # never dereferenced


@pytest.mark.parametrize("H", [-(2**63), -(2**63) + 1, -(2**62), -(2**62) - 1, 2**62, 2**62 + 1, 2**63 - 1, -1, 2**29 + 1])
def test_gate_refuses_widths_whose_double_wraps(H):
    L = mxq.Library().L
    assert L.mxq_silu_mul(FAKE, 0, 4, H, 64, FAKE, None) == INVALID
    assert L.mxq_fp8_silu_mul_1x128(FAKE, 0, 4, H, 64, FAKE, FAKE, None) == INVALID
    assert L.mxq_fp8_silu_mul_128x1(FAKE, 0, 4, H, 64, FAKE, FAKE, None) == INVALID
    assert L.mxq_silu_mul_grad(FAKE, FAKE, 0, 4, H, 64, 64, FAKE, None) == INVALID
