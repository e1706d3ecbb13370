"""The norm, the router, the gated activation and the dispatch of quantized
rows on the GPU, against 64-bit references from their definitions.

Tolerances, with u = 2^-24, the relative error of one fp32 rounding, and a
result of type t rounded by half a step, finfo(t).eps / 2, more.

* norm: a sum of K squares, all positive, in chains of at most K/256 + 80
  additions, is off by (K/256 + 80) u of itself, its root by half of that; the
  division, eps, root, reciprocal and two products add 8 u:
  (K/512 + 48) u |y|.
* its gradient: the mean over a row is off by (K/256 + 80) u of the mean of
  magnitudes, the other steps by 8 u of their terms; d_weight is a sum of rows/304
  terms and then of 304 in eight parts: (rows/304 + 60) u of the sum of magnitudes.
* gate: the exponential is off by 4 u (2^-22.5 of ex2.approx, and the
  correction's rounding), the sum and its reciprocal by 4 u, products by 4 u:
  16 u of the terms.  Results near the end of the range are off by its step.
* router: exponentials of differences up to d are off by (d + 4) u, sums of E
  terms by E u at most, divisions and products by 8 u.
* E4M3 payloads are rounded by 2^-4 of themselves, or by 2^-10 of their scale.
"""

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import layer_ref as ref
from tests import moe_block_ref as bref
from tests.gpu_util import Guarded, host_bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0**-24


@pytest.fixture(scope="module")
def mx():
    return mxq.library()


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def normal(rng, *shape):
    return rng.standard_normal(shape).astype(np.float32)


def dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def rows_of(a, dtype, ld=None, shift=0):
    """Device rows a with a stride of ld elements, `shift` elements behind an aligned address, NaN around them."""
    ld = ld or a.shape[1]
    base = torch.full((shift + a.shape[0] * ld,), float("nan"), dtype=dtype, device="cuda")
    t = base[shift:].view(a.shape[0], ld)[:, : a.shape[1]]
    t.copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return t


def near(got, want, tol):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    nan = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(got), nan)
    with np.errstate(invalid="ignore"):
        bad = ~nan & ~((np.abs(got - want) <= tol) | (got == want))
    assert not bad.any(), f"{bad.sum()} of {bad.size} off at {np.argwhere(bad)[:3].tolist()}: {got[bad][:3]} for {want[bad][:3]}"


def near_quantized(data, scales, want, rel, columns=False):
    """Payloads and codes of values that are `want` but for a relative error of rel."""
    d, c = host_bits(data), host_bits(scales).astype(np.int64)
    if columns:
        d, c, want = d.T, c.T, want.T
    d, c = d.reshape(want.shape), c.reshape(want.shape[0], -1)
    lo, hi = (ref.quant_rows(want * (1 + k * rel))[1].astype(np.int64) for k in (-1, 1))
    assert ((lo <= c) & (c <= hi)).all()
    code = np.repeat(c, 128, 1)[:, : want.shape[1]]
    nan = code == 255
    assert (d[nan] == 0x7F).all()
    scale = np.ldexp(1.0, np.minimum(code, 254) - 127)
    got = ref.e4m3_decode(d) * scale
    v = np.where(nan, 0.0, want)
    near(np.where(nan, 0.0, got), v, (2.0**-4 + 2 * rel) * np.abs(v) + 2.0**-10 * scale)


# ------------------------------------------------------------------- norm

# every form: a vector unit a thread, two, ragged and long rows, one element, a warp's and a block's edges
WIDTHS = [1, 16, 31, 128, 129, 512, 528, 1000, 2064, 4096, 7184, 8192, 8208, 8321, 16400, 20011, 33024]


def norm_rel(K):
    return (K / 512 + 48) * U


def check_norm(r, x, res, w, eps, dtype):
    h = f64(x) if res is None else f64((x.float() + res.float()).to(dtype))
    K = h.shape[1]
    y, rstd = bref.norm(h, f64(w), eps)
    if res is not None:
        np.testing.assert_array_equal(f64(r.h), h)
    near(r.rstd, rstd, norm_rel(K) * rstd)
    near(r.y, y, (norm_rel(K) + half_step(dtype)) * np.abs(y))
    near_quantized(r.data, r.scales, y, norm_rel(K))
    if dtype == F32:  # then y is what was quantized
        d, s = mxq.mxq_fp8_quant_1x128(r.y)
        np.testing.assert_array_equal(host_bits(r.data), host_bits(d))
        np.testing.assert_array_equal(host_bits(r.scales), host_bits(s))


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(mx, K, dtype, residual):
    rng = np.random.default_rng(K)
    rows = 5 if K > 9000 else 37
    size = np.exp2(rng.integers(-20, 20, (rows, 1)))
    x, w = dev(normal(rng, rows, K) * size, dtype), dev(1 + 0.3 * normal(rng, K), F32 if K % 3 else dtype)
    res = dev(normal(rng, rows, K) * size, dtype) if residual else None
    eps = 1e-5
    r = mx.rmsnorm(x, w, res, eps, normed=True, stats=True)
    check_norm(r, x, res, w, eps, dtype)
    # each output alone, between canaries, is the same
    data, scales, y, h = Guarded((rows, K), torch.uint8), Guarded(tuple(r.scales.shape), torch.uint8), Guarded((rows, K), dtype), Guarded((rows, K), dtype)
    mx.plan_rmsnorm(x, w, res, eps, data=data.t, scales=scales.t)()
    mx.plan_rmsnorm(x, w, res, eps, y=y.t)()
    rstd = Guarded((rows,), F32)
    mx.plan_rmsnorm(x, w, res, eps, rstd=rstd.t, h=h.t if residual else None)()
    for part, whole in ((data, r.data), (scales, r.scales), (y, r.y), (rstd, r.rstd)) + (((h, r.h),) if residual else ()):
        assert part.intact()
        np.testing.assert_array_equal(host_bits(part.t), host_bits(whole))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K,ld,shift", [(256, 272, 0), (256, 272, 16), (256, 270, 0), (256, 256, 1), (8, 24, 3), (4096, 4112, 16), (9000, 9001, 1)])
def test_norm_of_strided_rows_in_place(mx, dtype, K, ld, shift):
    rng = np.random.default_rng(K + ld)
    a, b = normal(rng, 9, K), normal(rng, 9, K)
    w = dev(normal(rng, K), dtype)
    x, res = rows_of(a, dtype, ld, shift), rows_of(b, dtype, ld, shift)
    r = mx.rmsnorm(x, w, res, normed=True, stats=True)
    check_norm(r, x, res, w, 1e-6, dtype)
    for over in range(2):
        pair = [rows_of(a, dtype, ld, shift), rows_of(b, dtype, ld, shift)]
        got = mx.rmsnorm(pair[0], w, pair[1], normed=True, stats=True, h=pair[over])
        for t, want in zip(got, r):
            assert torch.equal(t, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("K,ld,shift,rows", [(257, 257, 0, 1300), (383, 385, 3, 1220), (1000, 1000, 1, 1000), (1001, 1004, 5, 901), (4096, 4097, 0, 650), (7183, 7183, 0, 640),
                                             (8190, 8190, 1, 611), (8191, 8191, 7, 610), (8192, 8193, 1, 609)])
def test_norm_of_many_ragged_rows(mx, K, ld, shift, rows, dtype, residual):
    """Rows at every place of 16 bytes, as many as take turns on the device: what few of them give, bit for bit, and nothing beside it."""
    gen = torch.Generator("cuda").manual_seed(K)
    base = torch.full((2, shift + rows * ld), float("nan"), dtype=dtype, device="cuda")
    x, res = (b[shift:shift + rows * ld].view(rows, ld)[:, :K] for b in base)
    x.copy_(torch.randn(rows, K, device="cuda", generator=gen))
    res.copy_(torch.randn(rows, K, device="cuda", generator=gen))
    res = res if residual else None
    w = torch.randn(K, device="cuda", generator=gen).to(dtype if K % 2 else F32)
    nb = -(-K // 128)
    out = [Guarded((rows, K), torch.uint8), Guarded((rows, nb), torch.uint8), Guarded((rows, K), dtype), Guarded((rows,), F32)] + ([Guarded((rows, K), dtype)] if residual else [])
    names = ("data", "scales", "y", "rstd", "h")
    mx.plan_rmsnorm(x, w, res, 1e-5, **{n: o.t for n, o in zip(names, out)})()
    assert all(o.intact() for o in out)
    for a in range(0, rows, 200):
        part = slice(a, min(a + 200, rows))
        few = mx.rmsnorm(x[part], w, None if res is None else res[part], 1e-5, normed=True, stats=True)
        for n, o in zip(names, out):
            np.testing.assert_array_equal(host_bits(o.t[part]), host_bits(getattr(few, n)))
    check_norm(few, x[part], None if res is None else res[part], w, 1e-5, dtype)
    if residual:  # in place
        for over in (x, res):
            keep = over.clone()
            got = mx.rmsnorm(x, w, res, 1e-5, h=over)
            assert torch.equal(got.data, out[0].t) and torch.equal(got.scales, out[1].t) and torch.equal(over, out[4].t)
            over.copy_(keep)


def test_norm_in_place_over_x_and_over_the_residual(mx):
    rng = np.random.default_rng(5)
    for K in (1040, 1041, 9001):
        a, b, w = normal(rng, 6, K), normal(rng, 6, K), dev(normal(rng, K))
        want = mx.rmsnorm(dev(a), w, dev(b))
        for over in ("x", "residual"):
            x, res = dev(a), dev(b)
            h = x if over == "x" else res
            r = mx.rmsnorm(x, w, res, h=h)
            assert r.h is h
            for got, ref_ in zip((r.data, r.scales, r.h), (want.data, want.scales, want.h)):
                np.testing.assert_array_equal(host_bits(got), host_bits(ref_))


def test_norm_of_more_dimensions_and_of_nothing(mx):
    w = torch.ones(256, device="cuda", dtype=BF16)
    x = torch.randn(2, 3, 256, device="cuda").to(BF16)
    r = mx.rmsnorm(x, w, x, normed=True, stats=True)
    assert r.data.shape == r.y.shape == r.h.shape == (2, 3, 256) and r.scales.shape == (2, 3, 2) and r.rstd.shape == (2, 3)
    flat = mx.rmsnorm(x.view(6, 256), w, x.view(6, 256), normed=True, stats=True)
    assert torch.equal(flat.data.view(r.data.shape), r.data) and torch.equal(flat.y.view(r.y.shape), r.y)
    one = mx.rmsnorm(x[0, 0], w, stats=True)
    assert one.data.shape == (256,) and one.scales.shape == (2,) and one.rstd.shape == ()
    empty = mx.rmsnorm(x[:0], w, x[:0], normed=True, stats=True)
    assert empty.data.shape == (0, 3, 256) and empty.rstd.shape == (0, 3)
    d_h, d_w = mx.rmsnorm_grad(x[:0], x[:0], w, empty.rstd)
    assert d_h.shape == (0, 3, 256) and not d_w.any()


@pytest.mark.parametrize("K", [512, 519])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_zeros_nan_and_infinity(mx, dtype, K):
    x = torch.ones(6, K, device="cuda", dtype=dtype)
    x[0] = 0
    x[1, 3], x[2, K - 1], x[3, 5] = float("nan"), float("inf"), 3e38
    w = torch.ones(K, device="cuda", dtype=dtype)
    r = mx.rmsnorm(x, w, torch.zeros_like(x), 0.0, normed=True, stats=True)
    y = f64(r.y)
    assert np.isnan(y[0]).all() and np.isinf(f64(r.rstd)[0])  # 0 * inf: eps of zero and a row of zeros
    assert np.isnan(y[1]).all() and (host_bits(r.data)[1] == 0x7F).all() and (host_bits(r.scales)[1] == 255).all()
    assert np.isnan(y[2, K - 1]) and not y[2, : K - 1].any() and f64(r.rstd)[2] == 0
    assert not y[3].any()
    near(y[4:], np.ones((2, K)), norm_rel(K))
    canonical = 0x7FC0 if dtype == BF16 else 0x7FC00000
    assert (host_bits(r.y)[1] == canonical).all() and host_bits(r.h)[1, 3] == canonical
    assert (host_bits(r.scales)[4] == 119).all()
    zero = mx.rmsnorm(x[:1], w, eps=1e-6, normed=True)
    assert not zero.y.any() and not zero.data.any() and not zero.scales.any()


@pytest.mark.parametrize("K", [1, 16, 129, 512, 1000, 4096, 7184, 8208, 8321, 16384, 16400])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,more", [(1, True), (37, False), (700, True)])
def test_norm_gradient(mx, K, dtype, rows, more):
    if rows == 700 and K > 4096:
        rows = 310
    rng = np.random.default_rng(K + rows)
    h, g = dev(normal(rng, rows, K) * np.exp2(rng.integers(-8, 8, (rows, 1))), dtype), dev(normal(rng, rows, K), dtype)
    w, g_h = dev(1 + 0.3 * normal(rng, K), BF16 if K % 3 else dtype), dev(normal(rng, rows, K), dtype) if more else None
    rstd = mx.rmsnorm(h, w, stats=True, quantized=False).rstd
    d_h, d_w = Guarded((rows, K), dtype), Guarded((K,), F32)
    mx.plan_rmsnorm_grad(g, h, w, rstd, d_h.t, d_w.t, g_h)()
    assert d_h.intact() and d_w.intact()
    want, want_w, size = bref.norm_grad(f64(g), f64(h), f64(w), f64(rstd), None if g_h is None else f64(g_h))
    near(d_h.t, want, (K / 256 + 88) * U * size + half_step(dtype) * np.abs(want))
    near(d_w.t, want_w, (rows / 304 + 60) * U * np.abs(f64(g) * f64(h) * f64(rstd)[:, None]).sum(0))
    alone, none = mx.rmsnorm_grad(g, h, w, rstd, g_h, weight_grad=False)
    assert none is None and torch.equal(alone, d_h.t)
    # over each operand
    for over in ("g", "h", "g_h") if more else ("g", "h"):
        t = {"g": g.clone(), "h": h.clone(), "g_h": None if g_h is None else g_h.clone()}
        d, dw = mx.rmsnorm_grad(t["g"], t["h"], w, rstd, t["g_h"], d_h=t[over])
        assert d is t[over] and torch.equal(d, d_h.t) and torch.equal(dw, d_w.t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ld,shift", [(272, 0), (272, 16), (270, 0), (257, 1)])
def test_norm_gradient_of_strided_rows(mx, dtype, ld, shift):
    rng = np.random.default_rng(ld)
    a, b, c = (normal(rng, 50, 256) for _ in range(3))
    w = dev(normal(rng, 256), dtype)
    h, g, g_h = rows_of(a, dtype, ld, shift), rows_of(b, dtype, ld, shift), rows_of(c, dtype, ld, shift)
    rstd = mx.rmsnorm(h, w, stats=True).rstd
    d_h, d_w = mx.rmsnorm_grad(g, h, w, rstd, g_h)
    want, want_w, size = bref.norm_grad(f64(g), f64(h), f64(w), f64(rstd), f64(g_h))
    near(d_h, want, 89 * U * size + half_step(dtype) * np.abs(want))
    near(d_w, want_w, 61 * U * np.abs(f64(g) * f64(h) * f64(rstd)[:, None]).sum(0))


# ------------------------------------------------------------------- gate


def check_gate(mx, x):
    v, dtype = f64(x), x.dtype
    H = v.shape[1] // 2
    with np.errstate(invalid="ignore", over="ignore"):
        a = bref.gate(v)
        tiny = 2.0**-148 * (1 + np.abs(v[:, :H])) * (1 + np.abs(v[:, H:])) + (2.0**-134 if dtype == BF16 else 0)
        near(mx.silu_mul(x), a, 16 * U * np.abs(a) + half_step(dtype) * np.abs(a) + tiny)
    fine = np.where(np.isfinite(a), a, np.nan)
    near_quantized(*mx.fp8_silu_mul_1x128(x), fine, 16 * U)
    near_quantized(*mx.fp8_silu_mul_128x1(x), fine, 16 * U, columns=True)


@pytest.mark.parametrize("rows,H", [(1, 1), (1, 16), (37, 129), (5, 128), (128, 512), (129, 1000), (200, 1040), (257, 8), (3, 7184), (1, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate(mx, rows, H, dtype):
    rng = np.random.default_rng(rows + H)
    check_gate(mx, dev(normal(rng, rows, 2 * H) * np.exp2(rng.integers(-3, 4, (rows, 1))), dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,ld,shift", [(128, 272, 0), (128, 256, 16), (128, 258, 0), (136, 272, 8), (48, 97, 1)])
def test_gate_of_strided_rows(mx, dtype, H, ld, shift):
    rng = np.random.default_rng(H)
    x = rows_of(normal(rng, 130, 2 * H), dtype, ld, shift)
    check_gate(mx, x)
    g = rows_of(normal(rng, 130, H), dtype, ld, shift)
    want, size = bref.gate_grad(f64(g), f64(x))
    near(mx.silu_mul_grad(g, x), want, 16 * U * size + half_step(dtype) * np.abs(want))


def test_gate_over_the_whole_range(mx):
    """Every bf16 gate, the infinities and NaN among them."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(BF16)
    for dtype in (BF16, F32):
        x = torch.stack([bits, torch.full_like(bits, 1.5)], 1).to(dtype).view(512, 128, 2).transpose(1, 2).reshape(512, 256).contiguous()
        v = f64(x)
        gate = v[:, :128]
        with np.errstate(invalid="ignore"):
            want = np.where(np.isneginf(gate), np.nan, gate * bref.sigmoid(gate) * 1.5)
        got = f64(mx.silu_mul(x))
        top = float(torch.finfo(dtype).max)
        want = np.where(want > top, np.inf, want)  # 1.5 times the largest ones
        over = np.isinf(got) & (want > top * (1 - 2.0**-8))
        tiny = 2.0**-147 * (1 + np.abs(gate)) + (2.0**-134 if dtype == BF16 else 0)
        fine = np.isfinite(want) & ~over
        near(np.where(fine, got, 0.0), np.where(fine, want, 0.0), (16 * U + half_step(dtype)) * np.abs(np.where(fine, want, 0)) + np.where(fine, tiny, 0.0))
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))


@pytest.mark.parametrize("H", [256, 250])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gates_far_below_zero(mx, H, dtype):
    """Blocks of gates near the end of the exponential's range, next to factors that bring them back; gates beyond it and of
    the type's lowest value give zeros."""
    rng = np.random.default_rng(H)
    x = normal(rng, 384, 2 * H)
    x[:128, :H] = -rng.uniform(70, 87, (128, H))
    x[:128, H:] *= 1e30
    x[128:256, :H] = -rng.uniform(88, 100, (128, H))
    x[256:, :H] = np.where(rng.random((128, H)) < 0.5, -1e4, float(torch.finfo(dtype).min))
    x[256:, H:] *= 1e30
    x = dev(x, dtype)
    want = bref.gate(f64(x))
    for columns, (d, s) in ((False, mx.fp8_silu_mul_1x128(x)), (True, mx.fp8_silu_mul_128x1(x))):
        near_quantized(d[:128], s[: 1 if columns else 128], want[:128], 16 * U, columns)
        assert not (host_bits(d[256:]) & 0x7F).any()
        codes = host_bits(s).astype(np.int64)
        codes = codes[1:2].repeat(128, 0) if columns else codes[128:256].repeat(128, 1)[:, :H]
        got = ref.e4m3_decode(host_bits(d[128:256])) * np.ldexp(1.0, codes - 127)
        assert (np.abs(got - want[128:256]) <= 1.1e-36 * np.abs(f64(x)[128:256, H:]) + 2.0**-4 * np.abs(want[128:256]) + 2.0**-137).all()


@pytest.mark.parametrize("rows,H", [(1, 1), (1, 16), (37, 129), (128, 512), (129, 1000), (3, 7184)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_gradient(mx, rows, H, dtype):
    rng = np.random.default_rng(rows + H)
    x, g = dev(3 * normal(rng, rows, 2 * H), dtype), dev(normal(rng, rows, H), dtype)
    d = Guarded((rows, 2 * H), dtype)
    mx.plan_silu_mul_grad(g, x, d.t)()
    assert d.intact()
    want, size = bref.gate_grad(f64(g), f64(x))
    near(d.t, want, 16 * U * size + half_step(dtype) * np.abs(want))


@pytest.mark.parametrize("H", [128, 136, 65])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_writes_its_outputs_alone(mx, H, dtype):
    x = dev(normal(np.random.default_rng(H), 130, 2 * H), dtype)
    out = Guarded((130, H), dtype)
    mx.plan_silu_mul(x, out.t)()
    rows = Guarded((130, H), torch.uint8), Guarded((130, -(-H // 128)), torch.uint8)
    mx.plan_fp8_silu_mul_1x128(x, rows[0].t, rows[1].t)()
    columns = Guarded((130, H), torch.uint8), Guarded((2, H), torch.uint8)
    mx.plan_fp8_silu_mul_128x1(x, columns[0].t, columns[1].t)()
    assert all(g.intact() for g in (out,) + rows + columns)


@pytest.mark.parametrize("H", [256, 250])
def test_gate_poisons_the_blocks_of_nan_and_infinity(mx, H):
    x = torch.ones(130, 2 * H, device="cuda")
    x[3, 5], x[7, H + 140], x[129, 200] = float("nan"), float("inf"), float("-inf")
    d, s = mx.fp8_silu_mul_1x128(x)
    bad = np.zeros((130, 2), bool)
    bad[3, 0] = bad[7, 1] = bad[129, 1] = True
    np.testing.assert_array_equal(host_bits(s) == 255, bad)
    np.testing.assert_array_equal(host_bits(d) == 0x7F, np.repeat(bad, 128, 1)[:, :H])
    d, s = mx.fp8_silu_mul_128x1(x)
    bad = np.zeros((2, H), bool)
    bad[0, 5] = bad[0, 140] = bad[1, 200] = True
    np.testing.assert_array_equal(host_bits(s) == 255, bad)
    np.testing.assert_array_equal(host_bits(d) == 0x7F, np.repeat(bad, 128, 0)[:130])


# ------------------------------------------------------------------ router


def check_route(mx, logits, topk, bias=None, **kw):
    ids, w = mx.moe_route(logits, topk, bias=bias, **kw)
    x = f64(logits)
    want, want_w = bref.route(x, topk, None if bias is None else f64(bias), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    near(w, want_w, (x.shape[1] + 60) * U * np.abs(want_w) + 2.0**-140)


ROUTES = [
    dict(E=1, topk=1), dict(E=8, topk=8), dict(E=32, topk=2), dict(E=33, topk=32), dict(E=60, topk=4), dict(E=64, topk=6), dict(E=160, topk=6, groups=8, topk_groups=3),
    dict(E=128, topk=8, groups=4, topk_groups=2), dict(E=256, topk=8, groups=8, topk_groups=4, group_top=2), dict(E=72, topk=5, groups=3, topk_groups=2, group_top=2),
    dict(E=384, topk=8), dict(E=512, topk=10, groups=32, topk_groups=32, group_top=2), dict(E=1000, topk=3, groups=25, topk_groups=2, group_top=2), dict(E=1024, topk=32),
    dict(E=64, topk=2, groups=32, topk_groups=1, group_top=2), dict(E=32, topk=1, groups=32, topk_groups=3),
]


@pytest.mark.parametrize("route", ROUTES, ids=lambda r: "-".join(str(v) for v in r.values()))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route(mx, route, score, bias, dtype):
    kw = dict(route)
    E, topk = kw.pop("E"), kw.pop("topk")
    rng = np.random.default_rng(E + topk)
    logits, b = dev(2 * normal(rng, 301, E), dtype), dev(0.1 * normal(rng, E)) if bias else None
    for renormalize, scale in ((True, 1.0), (False, 2.5)):
        check_route(mx, logits, topk, b, score=score, renormalize=renormalize, scale=scale, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kw", [{}, dict(groups=4, topk_groups=2, group_top=2)])
def test_route_of_scores_that_32_bits_cannot_tell_apart(mx, score, kw):
    """A bias that takes each score to the same value but for its own rounding."""
    rng = np.random.default_rng(3)
    x = np.repeat(normal(rng, 1, 64), 40, 0)
    x[1:] += np.float32(1e-6) * normal(rng, 39, 64)
    bias = (0.7 - bref.scores(x[:1].astype(np.float64), score)[0]).astype(np.float32)
    check_route(mx, dev(x), 8, dev(bias), score=score, **kw)


def test_route_of_equal_logits_takes_the_lowest_index(mx):
    x = torch.zeros(7, 96, device="cuda")
    x[1], x[2, 90:], x[3, ::2], x[4] = -0.0, 1.0, -0.0, torch.finfo(F32).min
    x[5, ::3] = torch.finfo(F32).min
    for kw in (dict(), dict(bias=torch.full((96,), 0.25, device="cuda")), dict(groups=8, topk_groups=2, group_top=2), dict(groups=3, topk_groups=1)):
        for score in ("softmax", "sigmoid"):
            check_route(mx, x, 8, score=score, **kw)
            check_route(mx, x.to(BF16), 8, score=score, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_with_experts_out_of_service(mx, score):
    rng = np.random.default_rng(9)
    x = dev(normal(rng, 33, 64))
    x[:, 5] = x[:, 40:44] = -torch.inf
    x[3] = -torch.inf          # no expert at all
    x[4, 2:] = -torch.inf      # two
    x[5, :] = -torch.inf
    x[5, 63] = -1e30           # one, its score far below any other's range
    x[6] = -200.0              # scores that underflow
    x[6, 7] = -198.0
    bias = dev(0.1 * normal(rng, 64))
    for b in (None, bias, torch.where(torch.arange(64, device="cuda") % 3 == 0, -torch.inf, bias)):
        for kw in (dict(), dict(groups=8, topk_groups=3, group_top=2), dict(groups=8, topk_groups=3)):
            for renormalize in (True, False):
                check_route(mx, x, 6, b, score=score, renormalize=renormalize, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_rows_that_cannot_be_scored(mx, score):
    rng = np.random.default_rng(9)
    x = dev(normal(rng, 20, 70))
    x[2, 69], x[7, 0], x[11, 3] = float("nan"), float("inf"), float("-inf")
    check_route(mx, x, 5, score=score)
    check_route(mx, x, 5, dev(normal(rng, 70)), score=score)
    bias = dev(normal(rng, 70))
    bias[4] = float("nan")
    check_route(mx, x, 5, bias, score=score)
    bias[4] = float("inf")  # always chosen
    check_route(mx, x, 5, bias, score=score)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route_of_strided_logits_writes_its_outputs_alone(mx, dtype):
    x = rows_of(normal(np.random.default_rng(2), 45, 60), dtype, 67, 3)
    ids, w = Guarded((45, 4), torch.int32), Guarded((45, 4), F32)
    mx.plan_moe_route(x, 4, ids.t, w.t)()
    assert ids.intact() and w.intact()
    want, want_w = bref.route(f64(x), 4)
    np.testing.assert_array_equal(ids.t.cpu().numpy(), want)
    near(w.t, want_w, 120 * U * want_w)
    d = Guarded((45, 60), dtype)
    g = torch.ones(45, 4, device="cuda")
    mx.plan_moe_route_grad(g, x, ids.t, d.t, renormalize=False)()
    assert d.intact()


@pytest.mark.parametrize("E,topk", [(1, 1), (8, 8), (32, 2), (60, 4), (256, 8), (384, 8), (1000, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route_gradient(mx, E, topk, score, renormalize, dtype):
    rng = np.random.default_rng(E)
    x, g = dev(2 * normal(rng, 203, E), dtype), dev(normal(rng, 203, topk))
    ids = np.argsort(normal(rng, 203, E), axis=1)[:, :topk].astype(np.int32)
    ids[rng.random(ids.shape) < 0.1] = -1
    ids[3], ids[4, 0] = -1, E + 7
    if topk > 1:
        ids[5, 1] = ids[5, 0]  # one expert twice
    d = mx.moe_route_grad(g, x, dev(ids, torch.int32), score=score, renormalize=renormalize, scale=1.5)
    assert d.dtype == dtype
    want, size = bref.route_grad(f64(g), f64(x), ids, score, renormalize, 1.5)
    near(d, want, (E + 80) * U * size + half_step(dtype) * np.abs(want) + 2.0**-140)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E", [60, 64])
def test_route_gradient_of_nan_stays_in_its_row(mx, E, dtype):
    x, g = dev(normal(np.random.default_rng(E), 12, E), dtype), torch.ones(12, 3, device="cuda")
    ids = torch.arange(36, dtype=torch.int32, device="cuda").view(12, 3)
    x[2, 7], x[5, 15], g[8, 1] = float("nan"), float("nan"), float("nan")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            d = mx.moe_route_grad(g, x, ids, score=score, renormalize=renormalize)
            bad = torch.isnan(d).cpu()
            want = torch.zeros(12, E, dtype=torch.bool)
            for row in (2, 5, 8):  # softmax's sum takes it to all experts, a renormalised weight to the chosen ones
                if score == "softmax" and not renormalize:
                    want[row] = True
                elif renormalize:
                    want[row, 3 * row:3 * row + 3] = True
            want[2, 7] = want[5, 15] = want[8, 25] = True
            assert torch.equal(bad, want), (score, renormalize)
            if dtype == BF16:
                assert (host_bits(d)[want.numpy()] == 0x7FC0).all()


@pytest.mark.parametrize("T", [40, 16400])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_padded_rows(mx, T, score):
    """Rows of zeros and the rows between them, with the biases of a router that has not been balanced yet."""
    x = dev(normal(np.random.default_rng(T), T, 128))
    x[1::2] = 0.0
    for bias in (torch.zeros(128, device="cuda"), torch.full((128,), -0.25, device="cuda"), None):
        check_route(mx, x, 6, bias, score=score, groups=8, topk_groups=3, group_top=2)


def test_route_gradient_of_what_was_routed(mx):
    """Rows with few experts, or none, and scores that underflow have finite gradients; a token of one expert none."""
    x = torch.randn(9, 40, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[0] = -torch.inf
    x[1, 1:] = -torch.inf
    x[2] = -300.0
    x[2, 5] = -299.0
    x[3, 20:] = -torch.inf
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            ids, _ = mx.moe_route(x, 4, score=score, renormalize=renormalize)
            d = mx.moe_route_grad(torch.randn(9, 4, device="cuda"), x, ids, score=score, renormalize=renormalize)
            assert torch.isfinite(d).all() and not d[0].any() and not d[3, 20:].any()
            if renormalize:
                assert not d[1].any()


def test_route_of_no_tokens(mx):
    ids, w = mx.moe_route(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2)
    assert mx.moe_route_grad(w, torch.empty(0, 8, device="cuda"), ids).shape == (0, 8)


# ---------------------------------------------------------------- dispatch


@pytest.mark.parametrize("K,ld,shift", [(1, 1, 0), (128, 128, 0), (129, 131, 1), (7184, 7184, 0), (256, 272, 16), (260, 264, 4), (16, 33, 0)])
@pytest.mark.parametrize("align", [1, 128])
def test_dispatch_of_quantized_rows(mx, K, ld, shift, align):
    rng = np.random.default_rng(K)
    x = dev(normal(rng, 77, K))
    data, scales = mx.fp8_quant_1x128(x)
    rows = torch.full((shift + 77 * ld,), 0xA5, dtype=torch.uint8, device="cuda")[shift:].view(77, ld)[:, :K]
    rows.copy_(data)
    ids = dev(rng.integers(-1, 6, (77, 3)), torch.int32)
    source = mx.moe_sort(ids, 6, align).source
    want = mx.fp8_quant_1x128(x, index=source, index_div=3)
    out, codes = Guarded(tuple(want[0].shape), torch.uint8), Guarded(tuple(want[1].shape), torch.uint8)
    mx.plan_fp8_dispatch(rows, scales, source, 3, out.t, codes.t)()
    assert out.intact() and codes.intact() and torch.equal(out.t, want[0]) and torch.equal(codes.t, want[1])
    got = mx.fp8_dispatch(rows.view(torch.float8_e4m3fn), scales, source, 3)
    assert got[0].dtype == torch.float8_e4m3fn and torch.equal(got[0].view(torch.uint8), want[0])
    stray = dev(np.int32([0, 77 * 3, 2**31 - 1, -(2**31), 230]), torch.int32)  # choices that leave the tokens
    got = mx.fp8_dispatch(rows, scales, stray, 3)
    assert torch.equal(got[0][0], data[0]) and torch.equal(got[0][4], data[76]) and not got[0][1:4].any() and not got[1][1:4].any()


# ---------------------------------------------------- streams, graphs, runs


def small_run(mx, x, res, w, logits, bias, fc):
    """The serving path between the products, and what they are given."""
    r = mx.rmsnorm(x, w, res, normed=True, stats=True)
    ids, weights = mx.moe_route(logits, 2, bias=bias, score="sigmoid")
    order = mx.moe_sort(ids, logits.shape[1])
    q, c = mx.fp8_dispatch(r.data, r.scales, order.source, 2)
    a, ac = mx.fp8_silu_mul_1x128(fc)
    d_x = mx.silu_mul_grad(mx.silu_mul(fc), fc)
    d_l = mx.moe_route_grad(weights, logits, ids, score="sigmoid")
    d_h, d_w = mx.rmsnorm_grad(r.y, r.h, w, r.rstd, g_h=x)
    return [r.data, r.scales, r.y, r.h, r.rstd, ids, weights, q, c, a, ac, d_x, d_l, d_h, d_w]


def inputs(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return [new(96, 512).to(BF16), new(96, 512).to(BF16), new(512).to(BF16), new(96, 24), 0.1 * new(24), new(96, 1024).to(BF16)]


def test_a_captured_run_replays_on_new_inputs(mx):
    held = inputs(1)
    small_run(mx, *held)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = small_run(mx, *held)
    for seed in (2, 3):
        for a, b in zip(held, inputs(seed)):
            a.copy_(b)
        graph.replay()
        for got, want in zip(out, small_run(mx, *inputs(seed))):
            assert torch.equal(got, want)


def test_runs_on_another_stream_and_two_at_once(mx):
    want = [small_run(mx, *inputs(s)) for s in (4, 5)]
    sets = [inputs(s) for s in (4, 5)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = small_run(mx, *sets[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


def test_the_fast_math_build_gives_the_same(mx):
    fast = mxq.Library(fastmath=True)
    for a, b in zip(small_run(fast, *inputs(6)), small_run(mx, *inputs(6))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("size", [1.0, 1e-38, 1e-41])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_fast_math_build_gives_the_same_near_the_ends(mx, size, dtype):
    """Subnormal numbers too, by every kernel: many tokens and few, whole units and ragged rows."""
    fast = mxq.Library(fastmath=True)
    gen = torch.Generator("cuda").manual_seed(11)
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731

    def same(f):
        for a, b in zip(f(fast), f(mx)):
            np.testing.assert_array_equal(a.cpu() if a.dtype == torch.int32 else host_bits(a), b.cpu() if b.dtype == torch.int32 else host_bits(b))

    for T in (300, 16400):
        for E, bias, kw in ((256, True, dict(score="sigmoid", groups=8, topk_groups=4, group_top=2)), (256, False, {}), (64, False, dict(score="sigmoid")),
                            (160, True, dict(groups=8, topk_groups=2, renormalize=False)), (128, True, dict(score="sigmoid"))):
            x, b = (size * new(T, E)).to(dtype), 0.05 * size * new(E) if bias else None
            same(lambda m: m.moe_route(x, 8, bias=b, **kw))
    for K in (512, 511):
        x, w = (size * new(400, K)).to(dtype), new(K)
        x2 = torch.cat([size * new(400, K), 1e30 * new(400, K)], 1).to(dtype)
        r = mx.rmsnorm(x, w, x, stats=True)
        same(lambda m: [t for t in m.rmsnorm(x, w, x, normed=True, stats=True)] + list(m.rmsnorm_grad(x, r.h, w, r.rstd, g_h=x)))
        same(lambda m: [m.silu_mul(x2), *m.fp8_silu_mul_1x128(x2), *m.fp8_silu_mul_128x1(x2), m.silu_mul_grad(x, x2)])


# ------------------------------------------------- routers of many tokens

MANY = [
    dict(E=256, topk=8, score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, scale=2.5),
    dict(E=256, topk=8, score="softmax", renormalize=False),
    dict(E=256, topk=6, score="softmax", bias=True, groups=16, topk_groups=5, group_top=2),
    dict(E=256, topk=1, score="sigmoid", groups=4, topk_groups=1),
    dict(E=192, topk=7, score="sigmoid", bias=True),
    dict(E=160, topk=6, score="softmax", groups=10, topk_groups=3, renormalize=False),
    dict(E=132, topk=8, score="softmax", bias=True),
    dict(E=128, topk=8, score="softmax", bias=True),
    dict(E=128, topk=4, score="sigmoid", bias=True, groups=8, topk_groups=2, group_top=2),
    dict(E=128, topk=2, score="softmax", groups=4, topk_groups=2, group_top=2),
    dict(E=96, topk=5, score="sigmoid", renormalize=False),
    dict(E=64, topk=6, score="softmax"),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(str(v) for v in c.values()))
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route_of_many_tokens(mx, case, dtype):
    """Ordinary rows, and among them rows with experts out of service, ties, values that 32 bits cannot tell apart, NaN,
    infinities, and scores that underflow."""
    kw = dict(case)
    E, topk, bias = kw.pop("E"), kw.pop("topk"), kw.pop("bias", False)
    rng = np.random.default_rng(E + topk)
    T = 16389
    x = 1.5 * normal(rng, T, E)
    b = 0.05 * normal(rng, E) if bias else None
    x[5::97, ::3] = -np.inf
    x[7::97, 2:] = -np.inf
    x[9::97] = -np.inf
    x[11::97] = 0.25                                   # every expert alike
    x[13::97, : E // 2] = 2.0                          # many alike
    x[15::97, 4], x[17::97, E - 1], x[19::97, 1] = np.nan, np.inf, 3e38
    x[21::97] -= np.float32(500.0)
    x[23::97, 8:16] = 4.0 + 1e-6 * normal(rng, len(x[23::97]), 8)
    logits = dev(x, dtype)
    check_route(mx, logits, topk, None if b is None else dev(b), **kw)
    if bias:
        b[3::7] = -np.inf
        check_route(mx, logits, topk, dev(b), **kw)
        s = bref.scores(x[:1].astype(np.float64), kw.get("score", "softmax"))[0]
        near_ties = dev(np.repeat(x[:1], T, 0) + np.float32(1e-6) * normal(rng, T, E))
        check_route(mx, near_ties, topk, dev((0.7 - s).astype(np.float32)), **kw)


@pytest.mark.parametrize("E,groups,topk_groups", [(256, 8, 4), (256, 16, 3), (128, 4, 2), (128, 8, 7), (160, 5, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [40, 16389])
def test_route_of_groups_that_32_bits_cannot_tell_apart(mx, E, groups, topk_groups, score, T):
    """The last group that is kept and the first that is not differ by a few units of 2^-26 of a score, or less."""
    rng = np.random.default_rng(E + groups)
    x = (1.5 * normal(rng, T, E)).astype(np.float64)
    bias = 0.05 * normal(rng, E).astype(np.float64) if score == "sigmoid" else np.zeros(E)
    act = bref.sigmoid if score == "sigmoid" else np.exp
    c = (act(x) + bias).reshape(T, groups, -1)
    order = np.argsort(c, 2)
    two = np.take_along_axis(c, order[:, :, -2:], 2)
    rank = np.argsort(-two.sum(2), 1)
    rows = np.arange(0, T, 7)
    kept, out = rank[rows, topk_groups - 1], rank[rows, topk_groups]
    # the second largest of the group that is out makes its sum that of the other
    e = out * (E // groups) + order[rows, out, -2]
    s = two[rows, kept].sum(1) - two[rows, out, 1] - bias[e] + 2.0**-26 * rng.standard_normal(len(rows)) * (1 if score == "sigmoid" else 8)
    fine = (s > 0) & (s + bias[e] < two[rows, out, 1]) & ((s < 1) | (score == "softmax"))
    rows, e, s = rows[fine], e[fine], s[fine]
    x[rows, e] = np.log(s / (1 - s)) if score == "sigmoid" else np.log(s)
    assert len(rows) > 0
    kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_top=2)
    check_route(mx, dev(x), 6, dev(bias) if score == "sigmoid" else None, **kw)


def test_route_of_many_tokens_gives_what_few_do(mx):
    """A token's choice does not depend on how many there are with it."""
    x = torch.randn(20000, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    bias = 0.1 * torch.randn(256, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    kw = dict(bias=bias, score="sigmoid", groups=8, topk_groups=4, group_top=2)
    ids, w = mx.moe_route(x, 8, **kw)
    for a in range(0, 20000, 1000):
        i, v = mx.moe_route(x[a:a + 1000], 8, **kw)
        assert torch.equal(i, ids[a:a + 1000])
        near(v, f64(w[a:a + 1000]), 100 * U * f64(w[a:a + 1000]))


# ----------------------------------------------------- ends of the ranges


def test_offsets_beyond_32_bits(mx):
    """Tensors of more than 2^31 elements: their last rows are those of a small call."""
    rows, K = 262400, 8192
    x = torch.empty(rows, K, dtype=BF16, device="cuda")
    x[-300:] = torch.randn(300, K, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[:-300] = 1.0
    w = torch.ones(K, dtype=BF16, device="cuda")
    whole, few = mx.rmsnorm(x, w, stats=True), mx.rmsnorm(x[-300:], w, stats=True)
    for a, b in ((whole.data, few.data), (whole.scales, few.scales), (whole.rstd, few.rstd)):
        assert torch.equal(a[-300:], b)
    d, _ = mx.rmsnorm_grad(x, x, w, whole.rstd, weight_grad=False)
    assert torch.equal(d[-300:], mx.rmsnorm_grad(x[-300:], x[-300:], w, few.rstd, weight_grad=False)[0])
    source = torch.arange(rows - 1, rows - 301, -1, dtype=torch.int32, device="cuda")
    got = mx.fp8_dispatch(whole.data, whole.scales, source, 1)
    assert torch.equal(got[0], few.data.flip(0)) and torch.equal(got[1], few.scales.flip(0))
    del d, whole
    for f in (mx.fp8_silu_mul_1x128, mx.silu_mul, lambda t: mx.silu_mul_grad(t[:, : K // 2], t)):
        a, b = f(x), f(x[-300:])
        for p, q in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
            assert torch.equal(p[-300:], q)
    a, b = mx.fp8_silu_mul_128x1(x), mx.fp8_silu_mul_128x1(x[-256:])  # rows is a multiple of 128
    assert torch.equal(a[0][-256:], b[0]) and torch.equal(a[1][-2:], b[1])


def test_rows_of_no_elements(mx):
    x, w = torch.empty(3, 0, device="cuda"), torch.empty(0, device="cuda")
    r = mx.rmsnorm(x, w, stats=True, normed=True)
    assert r.data.shape == (3, 0) and r.scales.shape == (3, 0) and torch.isnan(r.rstd).all()
    d, dw = mx.rmsnorm_grad(x, x, w, r.rstd)
    assert d.shape == (3, 0) and dw.shape == (0,)
    assert mx.silu_mul(x).shape == (3, 0) and mx.fp8_silu_mul_128x1(x)[1].shape == (1, 0)


def test_refusals_of_the_binding(mx):
    x, w, res = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda"), torch.ones(4, 64, device="cuda", dtype=BF16)
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    g = torch.ones(4, 2, device="cuda")
    for f in (lambda: mx.rmsnorm(x, w[:63]), lambda: mx.rmsnorm(x, w.cpu()), lambda: mx.rmsnorm(x, w, res), lambda: mx.rmsnorm(x, w, x[:3]),
              lambda: mx.rmsnorm(x, w, eps=-1.0), lambda: mx.rmsnorm(x, w, eps=float("nan")), lambda: mx.rmsnorm(x, w, eps=1e39), lambda: mx.rmsnorm(x, w, h=x),
              lambda: mx.rmsnorm(x.t(), w[:4]), lambda: mx.rmsnorm(x, w.expand(2, 64)), lambda: mx.rmsnorm_grad(x, res, w, w[:4]),
              lambda: mx.rmsnorm_grad(x, x, w, w[:5]), lambda: mx.rmsnorm_grad(x, x, w, w[:4], g_h=x[:, :32]), lambda: mx.moe_route(x, 0), lambda: mx.moe_route(x, 33),
              lambda: mx.moe_route(x, 65), lambda: mx.moe_route(x, 2, score="tanh"), lambda: mx.moe_route(x, 2, groups=3), lambda: mx.moe_route(x, 2, groups=4, topk_groups=5),
              lambda: mx.moe_route(x, 8, groups=32), lambda: mx.moe_route(x, 2, group_top=3), lambda: mx.moe_route(x, 2, bias=w.cpu()), lambda: mx.moe_route(x, 2, bias=w[:5]),
              lambda: mx.moe_route(x, 2, scale=float("inf")), lambda: mx.moe_route(x[0], 2), lambda: mx.moe_route_grad(g, x, ids.long()), lambda: mx.moe_route_grad(g[:3], x, ids),
              lambda: mx.moe_route_grad(g, x, ids[:3]), lambda: mx.silu_mul(x[:, :63]), lambda: mx.silu_mul_grad(x, x), lambda: mx.silu_mul_grad(res[:, :32], x),
              lambda: mx.fp8_silu_mul_1x128(x, data=torch.empty(4, 31, dtype=torch.uint8, device="cuda")),
              lambda: mx.fp8_dispatch(x, x, ids.view(-1), 2), lambda: mx.fp8_dispatch(res.view(torch.uint8), ids.view(torch.uint8)[:, :1], ids.view(-1), 2)):
        with pytest.raises(ValueError):
            f()
    half = x.half()
    for f in (lambda: mx.rmsnorm(half, w), lambda: mx.rmsnorm(x, w.half()), lambda: mx.moe_route(half, 2), lambda: mx.silu_mul(half)):
        with pytest.raises(mxq.MXQError):
            f()
