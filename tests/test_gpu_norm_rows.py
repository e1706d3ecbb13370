"""The norm's weight gradient over many rows.  A persistent block to a
multiprocessor adds up every 152nd row, in chains of rows/152 (rows longer than
8192 that are not on 16 bytes: 304 of them, rows/304), and eight partial sums
of 19 of those blocks each: (rows/152 + 60) u of the sum of magnitudes."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests.test_gpu_moe_block import BF16, F32, U, f64, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,K", [(40000, 16), (20000, 512), (9000, 1001), (6000, 4100), (4000, 8192), (3000, 9001)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weight_gradient_over_many_rows(rows, K, dtype):
    gen = torch.Generator("cuda").manual_seed(rows)
    h = torch.rand(rows, K, device="cuda", generator=gen).to(dtype)  # of one sign: the sums grow
    g = torch.rand(rows, K, device="cuda", generator=gen).to(dtype)
    w = torch.ones(K, device="cuda")
    rstd = mxq.mxq_rmsnorm(h, w, stats=True, quantized=False).rstd
    _, d_w = mxq.mxq_rmsnorm_grad(g, h, w, rstd)
    want = (f64(g) * f64(h) * f64(rstd)[:, None]).sum(0)
    near(d_w, want, (rows / 152 + 60) * U * want)
    assert np.isfinite(want).all() and torch.equal(d_w, mxq.mxq_rmsnorm_grad(g, h, w, rstd)[1])
