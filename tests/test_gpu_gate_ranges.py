"""The gated activation on the GPU: gates far below zero beside large factors.
Tolerances as in test_gpu_moe_block, but where a test derives its own."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import moe_block_ref as bref
from tests.test_gpu_moe_block import BF16, F32, U, dev, f64, half_step, near, near_quantized, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    return mxq.library()


# Gates between 87 and 167 below zero: as test_gpu_moe_block's 16 U, and what a bf16 gate's exponential leaves out in the second
# order, (168 * 4.9e-6)^2 / 2 = 3.4e-7 = 6 U.
FAR = 22 * U


def far_gates(rng, rows, H, dtype):
    x = normal(rng, rows, 2 * H)
    x[:, :H] = -rng.uniform(80, 160, (rows, 1)) - rng.uniform(0, 7, (rows, H))
    # a gate of -160 leaves 2^-224 of the other factor: 2^127 of it is a number of 2^-97
    x[:, H:] = np.exp2(rng.uniform(-8, 0, (rows, H)) + 127) * np.sign(x[:, H:])
    return dev(x, dtype)


@pytest.mark.parametrize("H", [256, 250])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_gates_next_to_large_factors(mx, H, dtype):
    rng = np.random.default_rng(H)
    x = far_gates(rng, 256, H, dtype)
    want = bref.gate(f64(x))
    assert (np.abs(want) > 2.0**-120).all() and np.abs(want).max() > 100  # neither zeros nor subnormal
    near_quantized(*mx.fp8_silu_mul_1x128(x), want, FAR)
    near_quantized(*mx.fp8_silu_mul_128x1(x), want, FAR, columns=True)
    near(mx.silu_mul(x), want, (FAR + half_step(dtype)) * np.abs(want))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_far_gate(mx, dtype):
    """All bf16 gates from -60 to -200: up to -167 with the bits that they have, beyond it no more than 2.4e-71 of the other factor."""
    gate = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(BF16)
    gate = gate[(gate <= -60) & (gate >= -200)]
    up = float(np.float32(1.5 * 2.0**100))
    x = torch.stack([gate, torch.full_like(gate, up)], 1).to(dtype).contiguous()  # a row to each, H = 1
    v = f64(x)
    want = bref.gate(v)
    tol = np.where(v[:, :1] > -167.5, FAR * np.abs(want), 2.4e-71 * up)
    near(mx.silu_mul(x), want, tol + half_step(dtype) * np.abs(want) + (2.0**-134 if dtype == BF16 else 2.0**-149))
    d, s = mx.fp8_silu_mul_1x128(x)
    got = f64(d.view(torch.float8_e4m3fn).float()) * np.ldexp(1.0, f64(s).astype(np.int64) - 127)
    near(got, want, tol + (2.0**-4 + FAR) * np.abs(want) + 2.0**-137)


@pytest.mark.parametrize("H", [256, 250])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_plain_form_of_far_gates(mx, H, dtype):
    """Gates of -88 to -100 beside factors of 1e30: what fp32 holds of exp(gate) alone is a handful of bits."""
    rng = np.random.default_rng(H)
    x = normal(rng, 130, 2 * H)
    x[:, :H] = -rng.uniform(88, 100, (130, H))
    x[:, H:] = 1e30 * (np.abs(x[:, H:]) + 1)
    x = dev(x, dtype)
    want = bref.gate(f64(x))
    near(mx.silu_mul(x), want, (FAR + half_step(dtype)) * np.abs(want))
    near_quantized(*mx.fp8_silu_mul_1x128(x), want, FAR)
    near_quantized(*mx.fp8_silu_mul_128x1(x), want, FAR, columns=True)


@pytest.mark.parametrize("H", [32, 31])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinite_and_lowest_gates_in_every_form(mx, H, dtype):
    """silu(-inf) is NaN, silu(inf) infinite, and the lowest number gives zero: in every form but for +inf of bf16, which the FP8
    forms poison either way."""
    x = torch.full((4, 2 * H), 1.5, device="cuda", dtype=dtype)
    x[0, :H], x[1, :H], x[2, :H], x[3, :H] = float("inf"), float("-inf"), torch.finfo(dtype).min, torch.finfo(dtype).max
    a = f64(mx.silu_mul(x))
    assert (a[0] == np.inf).all() and np.isnan(a[1]).all() and (a[2] == 0).all() and (a[3] == np.inf).all()
    x[:, H:] = 0.5
    assert (f64(mx.silu_mul(x))[3] == 0.5 * float(torch.finfo(dtype).max)).all()
    codes = f64(mx.fp8_silu_mul_1x128(x)[1])
    assert (codes[:2] == 255).all() and (codes[2] == 0).all() and (codes[3] < 255).all()


def check_gate_gradient(mx, x, g, rel=FAR):
    """With gates down to -167 the bounds are those of the forms above: what is added to 1, up to 168 of it, is off by 4 U, and
    so are the sums that test_gpu_moe_block counts; results may be subnormal."""
    want, size = bref.gate_grad(f64(g), f64(x))
    top = float(torch.finfo(x.dtype).max)
    assert np.isfinite(size).all() and (np.abs(want) < top).all()
    near(mx.silu_mul_grad(g, x), want, rel * size + half_step(x.dtype) * np.abs(want) + (2.0**-133 if x.dtype == BF16 else 2.0**-148))


@pytest.mark.parametrize("H", [64, 61])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_gradient_of_factors_whose_product_overflows(mx, H, dtype):
    """The derivative of silu brings the product back: gates far below zero, and the place where the derivative is zero."""
    rng = np.random.default_rng(H)
    for lo, hi, size in ((86, 100, 66), (100, 130, 72), (130, 166, 90), (60, 86, 100), (10, 60, 62)):
        x, g = normal(rng, 40, 2 * H), normal(rng, 40, H)
        x[:, :H] = -rng.uniform(lo, hi, (40, H))
        x[:, H:] = np.sign(x[:, H:]) * np.exp2(rng.uniform(size - 3, size, (40, H)))
        g = np.sign(g) * np.exp2(rng.uniform(size - 3, size, (40, H)))
        check_gate_gradient(mx, dev(x, dtype), dev(g, dtype))
        # one of the factors large, the other small: their order does not matter
        x[:, H:] *= 2.0**20
        check_gate_gradient(mx, dev(x, dtype), dev(g * 2.0**-24, dtype))
        check_gate_gradient(mx, dev(np.concatenate([x[:, :H], g * 2.0**-24], 1), dtype), dev(x[:, H:], dtype))


@pytest.mark.parametrize("H", [64, 61])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_gradient_of_gates_that_give_zero(mx, H, dtype):
    """A derivative of zero is zero times any number: not NaN because the other factors' product overflows first."""
    x, g = torch.full((6, 2 * H), 1e30, device="cuda", dtype=dtype), torch.full((6, H), 1e30, device="cuda", dtype=dtype)
    for row, gate in enumerate((-250.0, -1e3, -1e30, torch.finfo(dtype).min, -250.0, -1e4)):
        x[row, :H] = gate
    x[4, H:], g[4] = 1e38, 1e9
    assert not mx.silu_mul_grad(g, x).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_gradient_over_the_whole_range(mx, dtype):
    """Every finite bf16 gate beside large, ordinary and small factors."""
    gate = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(BF16)
    gate = gate[torch.isfinite(gate.float()) & (gate > -167)]
    for u, s in ((1.5, 0.75), (2.0**20, 2.0**-30), (-(2.0**-60), 2.0**40), (1e-38, 1.25)):
        keep = gate[gate.double().abs() * max(abs(u), 1.0) * s < 1e38]
        x = torch.stack([keep, torch.full_like(keep, u)], 1).to(dtype).contiguous()
        check_gate_gradient(mx, x, torch.full((len(x), 1), s, device="cuda", dtype=dtype))
