"""The FP8 linear layer and the mixture-of-experts operators on the GPU,
against 64-bit references from their definitions.

Quantizing, sorting and gathering are compared exactly.  A product of depth D
is a sum of D terms in fp32, each addition off by at most one unit in the last
place, 2^-23, of a partial sum that S = sum |a_k| |b_k| bounds: D * 2^-23 * S,
plus the rounding of the result, 2^-8 (bf16) or 2^-23 (fp32) of it."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import layer_ref as ref
from tests.gpu_util import Guarded, dev_bf16, dev_f32, dev_input, host_bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ULP = {BF16: 2.0**-8, F32: 2.0**-23}


@pytest.fixture(scope="module")
def mx():
    return mxq.library()


def f64(t):
    return t.detach().double().cpu().numpy()


def bytes_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def as_f64(a):
    """Host input (bf16 bits or fp32) in 64 bits."""
    return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64) if a.dtype == np.uint16 else a.astype(np.float64)


def bf16_bits(a):
    return (np.ascontiguousarray(a, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def close(got, want, S, depth, dtype):
    got = f64(got)
    nan = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(got), nan)
    tol = depth * 2.0**-23 * S + ULP[dtype] * np.abs(want)
    off = np.abs(got - want)
    bad = ~nan & ~(off <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.where(nan, 0, off / np.maximum(tol, 1e-300)))} times the bound"


# ------------------------------------------------------------- quantizing


def quant_inputs():
    rng = np.random.default_rng(11)
    wide = (rng.standard_normal((130, 300)) * np.exp2(rng.integers(-140, 120, (130, 300)))).astype(np.float32)
    k = np.arange(-126, 120)
    edge = np.ldexp(np.float32(1.75), k).astype(np.float32)  # amax = 448 * 2^s, and its neighbours
    edges = np.zeros((len(k) * 3, 128), np.float32)
    edges[0::3, 5], edges[1::3, 5], edges[2::3, 5] = edge, np.nextafter(edge, np.float32(0)), np.nextafter(edge, np.float32(np.inf))
    edges[:, 7] = edges[:, 5] * np.float32(-0.0107421875)
    odd = rng.standard_normal((257, 131)).astype(np.float32)
    odd[3, 7], odd[200, 130], odd[130, 0] = np.nan, np.inf, -np.inf
    odd[5, :128] = 0.0
    odd[6] = -0.0
    tiny = (rng.integers(0, 1 << 12, (5, 200)).astype(np.uint32) | (rng.integers(0, 2, (5, 200)).astype(np.uint32) << 31)).view(np.float32)
    return {
        "every bf16": np.arange(65536, dtype=np.uint16).reshape(512, 128),
        "every bf16, shuffled": rng.permutation(65536).astype(np.uint16).reshape(256, 256),
        "wide": wide, "wide bf16": bf16_bits(wide), "edges": edges, "odd": odd, "odd bf16": bf16_bits(odd),
        "subnormal": tiny, "one": np.float32([[3.25]]), "row": rng.standard_normal((1, 1040)).astype(np.float32),
        "column": bf16_bits(rng.standard_normal((700, 1))), "many": bf16_bits(rng.standard_normal((129, 1024))),
    }


@pytest.mark.parametrize("name", list(quant_inputs()))
@pytest.mark.parametrize("columns", [False, True])
def test_quant_is_exact(mx, name, columns):
    x_np = quant_inputs()[name]
    rows, K = x_np.shape
    want = (ref.quant_columns if columns else ref.quant_rows)(as_f64(x_np))
    d = Guarded((rows, K), torch.uint8)
    s = Guarded(want[1].shape, torch.uint8)
    (mx.fp8_quant_128x1 if columns else mx.fp8_quant_1x128)(dev_input(x_np), data=d.t, scales=s.t)
    assert d.intact() and s.intact()
    np.testing.assert_array_equal(host_bits(s.t), want[1])
    np.testing.assert_array_equal(host_bits(d.t), want[0])


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K,ld,shift", [(257, 300, 1), (256, 272, 8), (1024, 1024, 0), (136, 140, 4)])
def test_quant_of_strided_and_gathered_rows(mx, columns, dtype, K, ld, shift):
    rng = np.random.default_rng(K + ld)
    base = torch.from_numpy(rng.standard_normal(97 * ld + shift).astype(np.float32)).to(dtype).cuda()
    x = base[shift:].view(97, ld)[:, :K]
    index = rng.integers(-1, 4 * 97 + 9, 333).astype(np.int32)
    index[:3] = -1, np.iinfo(np.int32).max, np.iinfo(np.int32).min
    f, g = (mx.fp8_quant_128x1, ref.quant_columns) if columns else (mx.fp8_quant_1x128, ref.quant_rows)
    for idx, div in ((None, 1), (bytes_dev(index), 4)):
        want = g(f64(x) if idx is None else ref.gather(f64(x), index, div))
        data, scales = f(x, index=idx, index_div=div)
        np.testing.assert_array_equal(host_bits(scales), want[1])
        np.testing.assert_array_equal(host_bits(data), want[0])


def test_quant_of_nothing(mx):
    d, s = mx.fp8_quant_1x128(torch.empty(0, 256, dtype=BF16, device="cuda"))
    assert d.shape == (0, 256) and s.shape == (0, 2)
    d, s = mx.fp8_quant_1x128(torch.empty(0, 256, device="cuda"), index=torch.full((3,), -1, dtype=torch.int32, device="cuda"))
    assert not d.any() and not s.any()


# ---------------------------------------------------------------- products


def make_rows(rng, rows, n):
    x = rng.standard_normal((rows, n)) * np.exp2(rng.integers(-6, 6, (rows, 1)))
    return ref.quant_rows(x.astype(np.float32).astype(np.float64))


def make_columns(rng, rows, n):
    return ref.quant_columns((rng.standard_normal((rows, n)) * np.exp2(rng.integers(-6, 6, (1, n)))).astype(np.float32).astype(np.float64))


def make_weight(rng, E, N, K):
    w = rng.integers(0, 127, (E, N, K)).astype(np.uint8) | (rng.integers(0, 2, (E, N, K)) << 7).astype(np.uint8)
    tile = np.exp2(rng.integers(-20, 0, (E, -(-N // 128), -(-K // 128)))).astype(np.float32)
    return w, tile


def operands(rng, direction, M, N, K):
    """(device arguments, a [m, d], b [n, d] in 64 bits)"""
    if direction == "wgrad":
        g, gs = make_columns(rng, M, N)
        x, xs = make_columns(rng, M, K)
        return tuple(map(bytes_dev, (g, gs, x, xs))), ref.decode_columns(g, gs).T, ref.decode_columns(x, xs).T
    x, xs = make_rows(rng, M, K if direction == "fwd" else N)
    w, tile = make_weight(rng, 1, N, K)
    wd = ref.decode_weight(w[0], tile[0])
    return tuple(map(bytes_dev, (x, xs, w[0], tile[0]))), ref.decode_rows(x, xs), wd if direction == "fwd" else wd.T


def call(mx, direction):
    return {"fwd": mx.fp8_matmul, "dgrad": mx.fp8_matmul_dgrad, "wgrad": mx.fp8_matmul_wgrad}[direction]


SIZES = [(1, 1, 1), (1, 128, 128), (1, 1024, 2048), (2, 300, 144), (3, 17, 33), (16, 256, 512), (17, 129, 1040), (33, 640, 384), (64, 200, 4112),
         (65, 1000, 96), (127, 129, 130), (128, 128, 128), (129, 257, 255), (200, 4112, 272), (256, 256, 256), (300, 96, 2064), (385, 784, 656),
         (513, 1040, 1552), (1100, 528, 912), (300, 4240, 8336), (4200, 272, 288), (8400, 160, 304), (20, 9000, 300), (3, 304, 33000)]


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product(mx, direction, M, N, K, dtype):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    args, a, b = operands(rng, direction, M, N, K)
    want, S = ref.product(a, b)
    out = Guarded(want.shape, dtype)
    call(mx, direction)(*args, out=out.t)
    assert out.intact()
    close(out.t, want, S, a.shape[1], dtype)


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("rows,features", [(257, 129), (273, 272), (383, 400), (384, 385), (641, 640), (2305, 2064), (2064, 2305), (2433, 2432)])
@pytest.mark.parametrize("depth", [144, 1040])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_with_few_tiles_in_the_last_round(mx, direction, rows, features, depth, dtype):
    """Tiles of 256x256 that are taken in halves: with a second half of nothing, of a column, of some and of all 128."""
    M, N, K = {"fwd": (rows, features, depth), "dgrad": (rows, depth, features), "wgrad": (depth, rows, features)}[direction]
    args, a, b = operands(np.random.default_rng(rows * 31 + features + depth), direction, M, N, K)
    want, S = ref.product(a, b)
    out = Guarded(want.shape, dtype)
    call(mx, direction)(*args, out=out.t)
    assert out.intact()
    close(out.t, want, S, depth, dtype)


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("shift,pad", [(0, 16), (16, 48), (1, 5), (0, 7), (8, 0)])
def test_product_of_strided_operands(mx, direction, shift, pad):
    rng = np.random.default_rng(shift * 100 + pad)
    M, N, K = 150, 272, 400
    (a, sa, b, sb), av, bv = operands(rng, direction, M, N, K)
    want, S = ref.product(av, bv)

    def strided(t):
        buf = torch.full((shift + t.shape[0] * (t.shape[1] + pad) + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        v = buf[shift:][: t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], t.shape[1] + pad)[:, : t.shape[1]]
        v.copy_(t)
        return v

    wide = torch.full((want.shape[0], want.shape[1] + 13), 7.0, dtype=BF16, device="cuda")
    call(mx, direction)(strided(a), sa, strided(b), sb, out=wide[:, 5:5 + want.shape[1]])
    close(wide[:, 5:5 + want.shape[1]], want, S, av.shape[1], BF16)
    assert (wide[:, :5] == 7).all() and (wide[:, 5 + want.shape[1]:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(5, 256, 1000), (260, 384, 640), (700, 512, 512)])
def test_poison_stays_in_its_row_and_tile(mx, M, N, K):
    rng = np.random.default_rng(M)
    x, xs = make_rows(rng, M, K)
    w, tile = make_weight(rng, 1, N, K)
    w, tile = w[0], tile[0]
    xs[2, 1] = 255                        # a poisoned activation block
    x[4, K - 1] = 0x7F                    # a payload NaN
    w[129, 3] = 0xFF                      # in the weight
    tile[0, 2] = 3.0                      # no power of two: the first 128 features
    want, S = ref.product(ref.decode_rows(x, xs), ref.decode_weight(w, tile))
    want[:, :128] = np.nan
    close(mx.fp8_matmul(*map(bytes_dev, (x, xs, w, tile)), out_dtype=F32), want, S, K, F32)


@pytest.mark.parametrize("bad", [0.0, -1.0, np.inf, np.nan, 1.5, 2.0**-140])
def test_tile_scales_that_are_no_power_of_two_give_nan(mx, bad):
    rng = np.random.default_rng(3)
    x, xs = make_rows(rng, 20, 256)
    w, tile = make_weight(rng, 1, 256, 256)
    tile[0, 1, 0] = bad
    y = f64(mx.fp8_matmul(*map(bytes_dev, (x, xs, w[0], tile[0]))))
    assert np.isfinite(y[:, :128]).all() and np.isnan(y[:, 128:]).all()


def test_extreme_scales(mx):
    """Scale codes at both ends: powers whose product is an ordinary number."""
    rng = np.random.default_rng(4)
    x, _ = make_rows(rng, 40, 256)
    w, _ = make_weight(rng, 1, 256, 256)
    for code, t in ((0, 2.0**119), (250, 2.0**-127), (1, 2.0**126), (254, 2.0**-126)):
        xs = np.full((40, 2), code, np.uint8)
        tile = np.full((2, 2), t, np.float32)
        want, S = ref.product(ref.decode_rows(x, xs), ref.decode_weight(w[0], tile))
        close(mx.fp8_matmul(*map(bytes_dev, (x, xs, w[0], tile)), out_dtype=F32), want, S, 256, F32)


def test_empty_products(mx):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    tile = torch.ones(2, 1, device="cuda")
    assert mx.fp8_matmul(u8(0, 128), u8(0, 1), u8(256, 128), tile).shape == (0, 256)
    y = mx.fp8_matmul_wgrad(u8(0, 64), u8(0, 64), u8(0, 32), u8(0, 32))
    assert y.shape == (64, 32) and not y.any()
    wide = torch.full((3, 9), 5.0, device="cuda")
    mx.fp8_matmul(u8(3, 0), u8(3, 0), u8(7, 0), torch.zeros(1, 0, device="cuda"), out=wide[:, 1:8], out_dtype=F32)
    assert not wide[:, 1:8].any() and (wide[:, 0] == 5).all() and (wide[:, 8] == 5).all()


def test_the_products_are_each_others_gradients(mx):
    """With small whole numbers every quantization and sum is exact, so the differences of the loss <g, x W^T> are the
    gradients' own, without an error."""
    rng = np.random.default_rng(5)
    M, N, K = 200, 144, 272
    whole = lambda *s: rng.integers(-4, 5, s).astype(np.float32)  # noqa: E731
    x, dx, g, w, dw = whole(M, K), whole(M, K), whole(M, N), whole(N, K), whole(N, K)

    def weight(a):
        return bytes_dev(ref.e4m3_encode(a.astype(np.float64))), torch.ones(-(-N // 128), -(-K // 128), device="cuda")

    def loss(x, w):
        q, s = mx.fp8_quant_1x128(dev_f32(x))
        return float((mx.fp8_matmul(q, s, *weight(w), out_dtype=F32).double() * dev_f32(g)).sum())

    gq, gs = mx.fp8_quant_1x128(dev_f32(g))
    d_x = f64(mx.fp8_matmul_dgrad(gq, gs, *weight(w), out_dtype=F32))
    gc, xc = mx.fp8_quant_128x1(dev_f32(g)), mx.fp8_quant_128x1(dev_f32(x))
    d_w = f64(mx.fp8_matmul_wgrad(*gc, *xc))
    assert loss(x + dx, w) - loss(x, w) == (d_x * dx).sum()
    assert loss(x, w + dw) - loss(x, w) == (d_w * dw).sum()


def test_products_of_one_call_do_not_vary(mx):
    rng = np.random.default_rng(6)
    for direction, size in (("fwd", (9, 1024, 4096)), ("fwd", (600, 1024, 4096)), ("wgrad", (4096, 300, 500))):
        args, *_ = operands(rng, direction, *size)
        first = call(mx, direction)(*args, out_dtype=F32)
        for _ in range(5):
            assert torch.equal(first, call(mx, direction)(*args, out_dtype=F32))


def test_on_another_stream_and_in_a_graph(mx):
    rng = np.random.default_rng(8)
    args, a, b = operands(rng, "fwd", 40, 512, 1040)
    want, S = ref.product(a, b)
    out = torch.zeros(40, 512, dtype=F32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.fp8_matmul(*args, out=out)
    torch.cuda.current_stream().wait_stream(side)
    close(out, want, S, 1040, F32)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mx.plan_fp8_matmul("fwd", *args, out)()
    graph.replay()
    torch.cuda.synchronize()
    close(out, want, S, 1040, F32)


def test_dependent_calls_in_a_row(mx):
    """Kernels start while the one in front of them in the stream is still running; a chain of dependent calls gives what the
    same calls give one at a time."""
    rng = np.random.default_rng(9)
    w = [tuple(map(bytes_dev, (a[0], t[0] * np.float32(2.0**-4)))) for a, t in (make_weight(rng, 1, 384, 384) for _ in range(4))]
    first = torch.from_numpy(rng.standard_normal((190, 384)).astype(np.float32)).to(BF16).cuda()
    ids = torch.from_numpy(rng.integers(0, 4, (190, 1)).astype(np.int32)).cuda()

    def chain(wait):
        x, seen = first, []
        for i in range(24):
            order = mx.moe_sort(ids, 4)
            wait()
            rows = mx.moe_dispatch(x, order.source, 1)
            wait()
            q, s = mx.fp8_quant_1x128(rows)
            wait()
            y = mx.fp8_matmul(q, s, *w[i % 4]) if i % 2 else mx.fp8_matmul_dgrad(q, s, *w[i % 4])
            wait()
            x = mx.moe_combine(y, order.slots)
            wait()
            x = torch.nn.functional.normalize(x.float(), dim=1).to(BF16)
            wait()
            seen.append(x)
        return torch.stack(seen)

    apart = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert torch.equal(chain(lambda: None), apart)


def test_more_outputs_than_32_bits_count(mx):
    M, N, K = 70001, 32784, 128  # 2.3e9 outputs
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randint(0, 127, (M, K), dtype=torch.uint8, device="cuda", generator=g)
    w = torch.randint(0, 127, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    xs = torch.full((M, 1), 120, dtype=torch.uint8, device="cuda")
    y = mx.fp8_matmul(x, xs, w, torch.full((257, 1), 2.0**-6, device="cuda"))
    rows = [0, 1, 255, 256, 32767, 65535, 65536, 69888, 70000]
    a = ref.e4m3_decode(x[rows].cpu().numpy()) * 2.0**-7
    want, S = ref.product(a, ref.e4m3_decode(w.cpu().numpy()) * 2.0**-6)
    close(y[rows], want, S, K, BF16)


def test_more_elements_than_32_bits_count(mx):
    T, H = 150001, 14336  # 2.15e9 elements
    x = torch.empty(T, H, dtype=BF16, device="cuda")
    x.view(torch.int16).random_(-(1 << 14), 1 << 14, generator=torch.Generator("cuda").manual_seed(2))
    rows = [0, 127, 74999, 149796, 149999, 150000]
    xr = f64(x[rows])
    d, s = mx.fp8_quant_1x128(x)
    want = ref.quant_rows(xr)
    np.testing.assert_array_equal(host_bits(d[rows]), want[0])
    np.testing.assert_array_equal(host_bits(s[rows]), want[1])
    d, s = mx.fp8_quant_128x1(x)
    tail = (T - 1) // 128 * 128
    want = ref.quant_columns(f64(x[tail:]))
    np.testing.assert_array_equal(host_bits(d[tail:]), want[0])
    np.testing.assert_array_equal(host_bits(s[-1:]), want[1])
    del d, s
    slots = torch.tensor([[150000], [-1], [149796]], dtype=torch.int32, device="cuda")
    np.testing.assert_array_equal(f64(mx.moe_combine(x, slots)), np.stack([xr[5], np.zeros(H), xr[3]]))
    source = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    source[150000] = 149999
    out = mx.moe_dispatch(x, source, 1)
    np.testing.assert_array_equal(f64(out[149999:]), np.stack([np.zeros(H), xr[4]]))


# ----------------------------------------------------------------- experts


GROUPS = [  # rows of each expert
    [5], [0, 0, 3, 0], [1, 1, 1, 1, 1], [130, 0, 1, 129, 16, 128, 17], [0, 0, 0], [300, 2, 260], [40] * 33, [1] + [0] * 60 + [700],
]


@pytest.mark.parametrize("direction", ["fwd", "dgrad"])
@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("N,K", [(272, 400), (128, 1040), (1000, 96), (160, 9000), (5000, 160)])
def test_grouped_product(mx, direction, counts, N, K):
    rng = np.random.default_rng(sum(counts) + N)
    E, front, behind = len(counts), 0, 7
    off = np.concatenate([[front], front + np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1]) + behind
    x, xs = make_rows(rng, M, K if direction == "fwd" else N)
    w, tile = make_weight(rng, E, N, K)
    av = ref.decode_rows(x, xs)
    n = N if direction == "fwd" else K
    want, S = np.zeros((M, n)), np.zeros((M, n))
    for e in range(E):
        wd = ref.decode_weight(w[e], tile[e])
        sl = slice(off[e], off[e + 1])
        want[sl], S[sl] = ref.product(av[sl], wd if direction == "fwd" else wd.T)
    # poison behind the last expert's rows must not leave them
    if behind:
        xs[off[-1]:] = 255
    for dtype in (BF16, F32):
        out = Guarded((M, n), dtype)
        call(mx, direction)(*map(bytes_dev, (x, xs, w, tile)), offsets=bytes_dev(off), out=out.t)
        assert out.intact()
        close(out.t, want, S, av.shape[1], dtype)


@pytest.mark.parametrize("direction", ["fwd", "dgrad"])
def test_a_poisoned_expert_stays_alone(mx, direction):
    rng = np.random.default_rng(21)
    N, K, off = 200, 176, np.int32([0, 3, 140, 150])
    x, xs = make_rows(rng, 150, K if direction == "fwd" else N)
    w, tile = make_weight(rng, 3, N, K)
    w[0], w[2] = 0x7F, 0xFF
    av = ref.decode_rows(x, xs)
    wd = ref.decode_weight(w[1], tile[1])
    want, S = ref.product(av, wd if direction == "fwd" else wd.T)
    want[:3] = want[140:] = np.nan
    close(call(mx, direction)(*map(bytes_dev, (x, xs, w, tile)), offsets=bytes_dev(off)), want, S, av.shape[1], BF16)


@pytest.mark.parametrize("off", [[5, 9, 30], [-7, 12, 9000], [20, 10, 30], [0, 64, 64], [64, 64, 64], [0, -5, -9]])
def test_offsets_are_clamped(mx, off):
    rng = np.random.default_rng(22)
    off = np.int32(off)
    M, N, K = 64, 144, 160
    x, xs = make_rows(rng, M, K)
    w, tile = make_weight(rng, 2, N, K)
    av, o = ref.decode_rows(x, xs), ref.clamp_offsets(off, M)
    want, S = np.zeros((M, N)), np.zeros((M, N))
    for e in range(2):
        want[o[e]:o[e + 1]], S[o[e]:o[e + 1]] = ref.product(av[o[e]:o[e + 1]], ref.decode_weight(w[e], tile[e]))
    close(mx.fp8_matmul(*map(bytes_dev, (x, xs, w, tile)), offsets=bytes_dev(off), out_dtype=F32), want, S, K, F32)


@pytest.mark.parametrize("counts", [[128], [0, 256, 0, 128], [1, 130, 5, 128], [0, 0], [700, 3], [5000, 130, 0, 9300]])
@pytest.mark.parametrize("N,K", [(144, 272), (128, 128), (300, 97)])
def test_grouped_weight_gradient(mx, counts, N, K):
    rng = np.random.default_rng(sum(counts) + N)
    E = len(counts)
    room = [-(-c // 128) * 128 for c in counts]
    off = np.concatenate([[0], np.cumsum(room)]).astype(np.int32)
    M = int(off[-1]) + 70
    real = np.zeros(M, bool)
    for e in range(E):
        real[off[e]:off[e] + counts[e]] = True
    real[off[-1]:] = True  # rows behind the last expert count for none
    gv = rng.standard_normal((M, N)).astype(np.float32) * real[:, None]
    xv = rng.standard_normal((M, K)).astype(np.float32) * real[:, None]
    g, gs = ref.quant_columns(gv.astype(np.float64))
    x, xs = ref.quant_columns(xv.astype(np.float64))
    gd, xd = ref.decode_columns(g, gs), ref.decode_columns(x, xs)
    if M > off[-1]:
        gs[off[-1] // 128:] = 255
    want, S = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e in range(E):
        want[e], S[e] = ref.product(gd[off[e]:off[e + 1]].T, xd[off[e]:off[e + 1]].T)
    for dtype in (BF16, F32):
        out = Guarded((E, N, K), dtype)
        mx.fp8_matmul_wgrad(*map(bytes_dev, (g, gs, x, xs)), offsets=bytes_dev(off), out=out.t)
        assert out.intact()
        close(out.t, want, S, max(room), dtype)


@pytest.mark.parametrize("off", [[0, 200, 200], [0, 128, 200], [0, 0, 999], [-4, 100, 150]])
def test_grouped_weight_gradient_clamps_and_rounds_offsets(mx, off):
    rng = np.random.default_rng(23)
    M, N, K = 200, 136, 140
    g, gs = make_columns(rng, M, N)
    x, xs = make_columns(rng, M, K)
    gd, xd = ref.decode_columns(g, gs), ref.decode_columns(x, xs)
    o = np.minimum(-(-ref.clamp_offsets(np.array(off), M) // 128) * 128, M)
    want, S = np.zeros((2, N, K)), np.zeros((2, N, K))
    for e in range(2):
        want[e], S[e] = ref.product(gd[o[e]:o[e + 1]].T, xd[o[e]:o[e + 1]].T)
    close(mx.fp8_matmul_wgrad(*map(bytes_dev, (g, gs, x, xs)), offsets=bytes_dev(np.int32(off))), want, S, M, F32)


# -------------------------------------------------------------------- sort


@pytest.mark.parametrize("T,topk,E,align", [(1, 1, 1, 1), (1, 2, 32, 1), (31, 1, 2, 1), (48, 2, 32, 1), (33, 3, 33, 128), (512, 8, 256, 1),
                                            (4095, 1, 7, 128), (4096, 1, 7, 1), (4097, 1, 2048, 1), (3000, 6, 64, 100), (20000, 4, 256, 128)])
@pytest.mark.parametrize("kind", ["random", "dropped", "one expert", "none"])
def test_sort(mx, T, topk, E, align, kind):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, topk)).astype(np.int32)
    if kind == "dropped":
        ids = rng.integers(-3, E + 5, (T, topk)).astype(np.int32)
        ids[0, 0] = np.iinfo(np.int32).max
    elif kind == "one expert":
        ids[:] = E - 1
    elif kind == "none":
        ids[:] = -1
    want = ref.moe_sort(ids, E, align)
    got = mx.moe_sort(bytes_dev(ids), E, align)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


def test_sort_of_nothing(mx):
    order = mx.moe_sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert order.offsets.tolist() == [0] * 10 and order.source.numel() == 0 and order.slots.shape == (0, 4)


# -------------------------------------------------------------------- rows


def routed(mx, rng, T, topk, E, align):
    ids = rng.integers(-1, E, (T, topk)).astype(np.int32)
    order = mx.moe_sort(bytes_dev(ids), E, align)
    return order, order.source.cpu().numpy().astype(np.int64), order.slots.cpu().numpy().astype(np.int64)


def rows_view(rng, rows, H, dtype, pad):
    t = torch.from_numpy(rng.standard_normal((rows, H + pad)).astype(np.float32)).to(dtype).cuda()
    return t[:, pad // 2:pad // 2 + H] if pad else t


ROWS = [(1, 1, 1, 1, 1, 0), (7, 2, 4, 33, 1, 0), (48, 2, 32, 7184, 1, 0), (65, 4, 8, 256, 128, 0), (30, 8, 16, 1000, 1, 6), (129, 1, 3, 4100, 16, 8), (9, 3, 5, 520, 1, 3)]


@pytest.mark.parametrize("T,topk,E,H,align,pad", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dispatch_and_combine(mx, T, topk, E, H, align, pad, dtype):
    rng = np.random.default_rng(T * H)
    order, source, slots = routed(mx, rng, T, topk, E, align)
    x = rows_view(rng, T, H, dtype, pad)
    out = Guarded((len(source), H), dtype)
    mx.moe_dispatch(x, order.source, topk, out=out.t)
    assert out.intact()
    np.testing.assert_array_equal(f64(out.t), ref.gather(f64(x), source, topk))

    y = rows_view(rng, len(source), H, dtype, pad)
    y[torch.from_numpy(source < 0).cuda()] = float("nan")  # rows of no choice are not read
    w = torch.from_numpy(rng.random((T, topk)).astype(np.float32)).cuda()
    there = slots >= 0
    yv = np.where(there[..., None], f64(y)[np.maximum(slots, 0)], 0.0)
    for weights in (w, None):
        terms = yv * (f64(w)[..., None] if weights is not None else 1.0)
        out = Guarded((T, H), dtype)
        mx.moe_combine(y, order.slots, weights, out=out.t)
        assert out.intact()
        close(out.t, terms.sum(1), np.abs(terms).sum(1), topk, dtype)


@pytest.mark.parametrize("T,topk,E,H,align,pad", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_gradient(mx, T, topk, E, H, align, pad, dtype):
    rng = np.random.default_rng(T * H + 1)
    order, source, slots = routed(mx, rng, T, topk, E, align)
    y, g = rows_view(rng, len(source), H, dtype, pad), rows_view(rng, T, H, dtype, pad)
    y[torch.from_numpy(source < 0).cuda()] = float("nan")
    w = torch.from_numpy(rng.random((T, topk)).astype(np.float32)).cuda()
    d_rows, d_w = Guarded((len(source), H), dtype), Guarded((T, topk), F32)
    mx.plan_moe_combine_grad(g, y, order.source, order.slots, w, d_rows.t, d_w.t)()
    assert d_rows.intact() and d_w.intact()
    there = slots >= 0
    yv = np.where(there[..., None], f64(y)[np.maximum(slots, 0)], 0.0)
    terms = yv * f64(g)[:, None]
    close(d_w.t, terms.sum(2), np.abs(terms).sum(2), H, F32)
    want = np.zeros((len(source), H))
    want[slots[there]] = (f64(w)[..., None] * f64(g)[:, None])[there]
    close(d_rows.t, want, np.abs(want), 1, dtype)


def test_combine_gradient_against_differences(mx):
    """With weights that are eighths and rows of small whole numbers every sum is exact, so the differences of <g, combine> are
    the gradients' own."""
    rng = np.random.default_rng(31)
    T, topk, H = 50, 3, 72
    order, source, _ = routed(mx, rng, T, topk, 6, 1)
    whole = lambda *s: torch.from_numpy(rng.integers(-4, 5, s).astype(np.float32)).cuda()  # noqa: E731
    y, dy, g, w, dw = whole(len(source), H), whole(len(source), H), whole(T, H), whole(T, topk) / 8, whole(T, topk) / 8
    dy[order.source < 0] = 0
    loss = lambda y, w: float((mx.moe_combine(y, order.slots, w).double() * g).sum())  # noqa: E731
    d_rows, d_w = mx.moe_combine_grad(g, y, order.source, order.slots, w)
    assert loss(y + dy, w) - loss(y, w) == float((d_rows.double() * dy).sum())
    assert loss(y, w + dw) - loss(y, w) == float((d_w.double() * dw).sum())
    x, dx = whole(T, H), whole(T, H)
    back = mx.moe_combine(y, order.slots)
    sent = lambda x: float((mx.moe_dispatch(x, order.source, topk).double() * torch.where(order.source[:, None] >= 0, y, 0.0)).sum())  # noqa: E731
    assert sent(x + dx) - sent(x) == float((back.double() * dx).sum())


def test_slots_that_leave_the_rows_add_nothing(mx):
    y = torch.ones(4, 8, device="cuda")
    slots = torch.tensor([[0, 4], [-1, 1 << 30], [3, -(1 << 31)]], dtype=torch.int32, device="cuda")
    assert mx.moe_combine(y, slots)[:, 0].tolist() == [1.0, 0.0, 1.0]
    assert mx.moe_dispatch(y, torch.tensor([8, 7, -1], dtype=torch.int32, device="cuda"), 2)[:, 0].tolist() == [0.0, 1.0, 0.0]


# ---------------------------------------------------------------- refusals


def test_refusals(mx):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    x, xs, w, t = u8(40, 256), u8(40, 2), u8(384, 256), f32(3, 2)
    mx.fp8_matmul(x, xs, w, t)
    for bad in (
        lambda: mx.fp8_matmul(x, u8(40, 1), w, t),                            # scales of another size
        lambda: mx.fp8_matmul(x, xs.float(), w, t),                           # ... or type
        lambda: mx.fp8_matmul(x, u8(40, 4)[:, ::2], w, t),                    # ... or not contiguous
        lambda: mx.fp8_matmul(x, xs, w, f32(3, 1)),
        lambda: mx.fp8_matmul(x, xs, w, t.double()),
        lambda: mx.fp8_matmul(x, xs, u8(384, 128), t),                        # inner sizes
        lambda: mx.fp8_matmul(x.to(BF16), xs, w, t),                          # no payload bytes
        lambda: mx.fp8_matmul(x, xs, w.float(), t),
        lambda: mx.fp8_matmul(x[:1].expand(40, 256), xs, w, t),               # rows that overlap
        lambda: mx.fp8_matmul(x.t(), xs, w, t),
        lambda: mx.fp8_matmul(x, xs, w, t, out=f32(40, 383)),
        lambda: mx.fp8_matmul(x, xs, w, t, out=torch.zeros(40, 384)),         # on the CPU
        lambda: mx.fp8_matmul(x.cpu(), xs, w, t),
        lambda: mx.fp8_matmul(x, xs, w, t, offsets=i32(2)),                   # offsets without a stack
        lambda: mx.fp8_matmul(x, xs, w.view(1, 384, 256), t),                 # a stack without offsets
        lambda: mx.fp8_matmul(x, xs, w.view(1, 384, 256), t, offsets=i32(3)),
        lambda: mx.fp8_matmul(x, xs, w.view(1, 384, 256), t, offsets=i32(2).long()),
        lambda: mx.fp8_matmul(x, xs, w.view(1, 384, 256), t, offsets=i32(0)),
        lambda: mx.fp8_matmul_wgrad(x, u8(1, 256), u8(41, 256), u8(1, 256)),  # rows
        lambda: mx.fp8_matmul_wgrad(x, xs, x, u8(1, 256)),
        lambda: mx.plan_fp8_matmul("forward", x, xs, w, t, f32(40, 384)),
        lambda: mx.fp8_quant_1x128(f32(8, 4).t()),
        lambda: mx.fp8_quant_1x128(f32(4, 8), index=i32(3).long()),
        lambda: mx.fp8_quant_1x128(f32(4, 8), data=u8(4, 7)),
        lambda: mx.fp8_quant_128x1(f32(4, 8), scales=u8(2, 8)),
        lambda: mx.moe_sort(i32(8), 3),
        lambda: mx.moe_sort(i32(8, 2).long(), 3),
        lambda: mx.moe_sort(i32(8, 2), 0),
        lambda: mx.moe_sort(i32(8, 2), 3, align=0),
        lambda: mx.moe_sort(i32(8, 4)[:, ::2], 3),
        lambda: mx.moe_dispatch(f32(4, 8), i32(4).long(), 1),
        lambda: mx.moe_dispatch(f32(4, 8), i32(4), 1, out=f32(4, 7)),
        lambda: mx.moe_dispatch(f32(4, 8, 1), i32(4), 1),
        lambda: mx.moe_combine(f32(4, 8), i32(4)),
        lambda: mx.moe_combine(f32(4, 8), i32(4, 2), f32(4, 1)),
        lambda: mx.moe_combine(f32(4, 8), i32(4, 2), f32(4, 2).double()),
        lambda: mx.moe_combine_grad(f32(4, 8), f32(6, 8), i32(5), i32(4, 2), f32(4, 2)),
        lambda: mx.moe_combine_grad(f32(4, 8).to(BF16), f32(6, 8), i32(6), i32(4, 2), f32(4, 2)),
    ):
        with pytest.raises(ValueError):
            bad()
    for bad, status in (
        (lambda: mx.fp8_quant_1x128(f32(4, 8).half()), 2),
        (lambda: mx.fp8_matmul(x, xs, w, t, out_dtype=torch.float16), 2),
        (lambda: mx.moe_combine(f32(4, 8).half(), i32(4, 2)), 2),
        (lambda: mx.fp8_quant_1x128(f32(4, 8), index=i32(3), index_div=0), 1),
        (lambda: mx.moe_sort(i32(8, 2), 2049), 1),
        (lambda: mx.moe_dispatch(f32(4, 8), i32(4), 0), 1),
        (lambda: mx.fp8_matmul(x, xs, u8(1025, 384, 256), f32(1025, 3, 2), offsets=i32(1026)), 1),
    ):
        with pytest.raises(mxq.MXQError) as e:
            bad()
        assert e.value.status == status
