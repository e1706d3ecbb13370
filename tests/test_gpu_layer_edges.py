"""The FP8 linear layer and the mixture-of-experts operators at the ends of their
ranges, against 64-bit references from their definitions."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    return mxq.library()


def test_a_part_of_the_sort_that_ends_at_the_last_32_bit_row(mx):
    """One choice whose part is rounded up to 2^31 - 1 rows: every row behind it is -1, and none in front of the order or behind
    it is touched."""
    rows, edge, canary = (1 << 31) - 1, 1024, 7
    room = torch.full((rows + 2 * edge,), canary, dtype=torch.int32, device="cuda")
    source = room[edge:edge + rows]
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    order = mxq.MoeOrder(i32(2), source, i32(1, 1))
    mx.plan_moe_sort(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1, order, align=rows)()
    assert order.offsets.tolist() == [0, rows] and order.slots.tolist() == [[0]]
    assert int(source[0]) == 0
    assert (room[:edge] == canary).all() and (room[edge + rows:] == canary).all()
    for piece in source[1:].split(1 << 28):
        assert (piece == -1).all()
