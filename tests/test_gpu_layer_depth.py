"""Deep products of the FP8 linear layer.

With small whole numbers and scales of a few powers of two every partial sum
is a whole number below 2^24, which neither a rounding nor a truncation
changes: the result is exact, and a block, a group of scales, a segment or a
share of the depth that is lost, doubled or scaled wrongly shows as itself.

With normally distributed operands the error of an fp32 result is measured
against its norm.  A sum over the whole depth that cuts off what 24 bits
cannot hold has an error in proportion to the depth, about 2.5e-7 of the norm
at 4608 and so 1.8e-6 at 33000; summed in segments it stays below 1e-6.  A
bf16 result's own rounding is at most 2^-9 of each value, and its sum, which is
not cut into segments, off by less than 1e-5 at these depths."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import layer_ref as ref
from tests.test_gpu_layer import BF16, F32, bytes_dev, call, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    return mxq.library()


def sizes(direction, rows, features, depth):
    """M, N, K of a product with that many output rows and columns."""
    return {"fwd": (rows, features, depth), "dgrad": (rows, depth, features), "wgrad": (depth, rows, features)}[direction]


def whole_rows(rng, rows, n):
    return (ref.e4m3_encode(rng.integers(-4, 5, (rows, n)).astype(np.float64)),
            (127 + rng.integers(0, 3, (rows, -(-n // 128)))).astype(np.uint8))


def whole_columns(rng, rows, n):
    return (ref.e4m3_encode(rng.integers(-4, 5, (rows, n)).astype(np.float64)),
            (127 + rng.integers(0, 3, (-(-rows // 128), n))).astype(np.uint8))


def whole_weight(rng, *shape):
    tiles = shape[:-2] + (-(-shape[-2] // 128), -(-shape[-1] // 128))
    return (ref.e4m3_encode(rng.integers(-4, 5, shape).astype(np.float64)),
            np.exp2(rng.integers(0, 3, tiles)).astype(np.float32))


def check_exact(ys, a, b):
    """Each y is a b^T, rounded to nearest even where it is bf16."""
    want, S = ref.product(a, b)
    assert S.max(initial=0) < 1 << 24  # so every partial sum is below it
    want = torch.from_numpy(want).to(F32)  # exact
    for y in ys:
        np.testing.assert_array_equal(f64(y), want.to(y.dtype).double().numpy())


DEEP = [  # output rows, columns, depth
    (1, 300, 2048), (1, 130, 8192), (3, 304, 33000), (20, 500, 9000), (40, 260, 5000), (100, 400, 4096), (200, 1040, 4736), (2, 130, 40000),
    (300, 600, 9216), (513, 272, 4736), (300, 304, 33000), (600, 520, 4608), (257, 129, 4609), (2433, 304, 1040),
]


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("rows,features,depth", DEEP)
def test_whole_numbers_are_exact(mx, direction, rows, features, depth):
    rng = np.random.default_rng(rows + 3 * features + 7 * depth)
    M, N, K = sizes(direction, rows, features, depth)
    if direction == "wgrad":
        p, q = whole_columns(rng, M, N), whole_columns(rng, M, K)
        a, b = ref.decode_columns(*p).T, ref.decode_columns(*q).T
    else:
        p, q = whole_rows(rng, M, K if direction == "fwd" else N), whole_weight(rng, N, K)
        a, b = ref.decode_rows(*p), ref.decode_weight(*q)
        b = b if direction == "fwd" else b.T
    args = tuple(map(bytes_dev, (*p, *q)))
    outs = [torch.full((rows, features + pad), 7.0, dtype=dtype, device="cuda") for dtype in (BF16, F32) for pad in (0, 3)]
    for wide in outs:
        call(mx, direction)(*args, out=wide[:, :features])
        assert (wide[:, features:] == 7).all()
    check_exact([wide[:, :features] for wide in outs], a, b)


@pytest.mark.parametrize("direction", ["fwd", "dgrad"])
@pytest.mark.parametrize("counts", [[3, 0, 1, 20], [300, 0, 17, 130, 60]])
@pytest.mark.parametrize("features,depth", [(272, 4736), (200, 9216)])
def test_whole_numbers_per_expert_are_exact(mx, direction, counts, features, depth):
    rng = np.random.default_rng(sum(counts) + depth)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, N, K = sizes(direction, int(off[-1]), features, depth)
    p, q = whole_rows(rng, M, K if direction == "fwd" else N), whole_weight(rng, len(counts), N, K)
    ys = [call(mx, direction)(*map(bytes_dev, (*p, *q)), offsets=bytes_dev(off), out_dtype=dtype) for dtype in (BF16, F32)]
    a, b = ref.decode_rows(*p), ref.decode_weight(*q)
    for e in range(len(counts)):
        check_exact([y[off[e]:off[e + 1]] for y in ys], a[off[e]:off[e + 1]], b[e] if direction == "fwd" else b[e].T)


@pytest.mark.parametrize("rooms", [[128, 0, 4736], [0, 9216, 128, 33024, 256]])
@pytest.mark.parametrize("N,K", [(144, 272), (300, 97)])
def test_whole_numbers_of_an_experts_weight_gradient_are_exact(mx, rooms, N, K):
    rng = np.random.default_rng(sum(rooms) + N)
    off = np.concatenate([[0], np.cumsum(rooms)]).astype(np.int32)
    M = int(off[-1]) + 70
    p, q = whole_columns(rng, M, N), whole_columns(rng, M, K)
    ys = [mx.fp8_matmul_wgrad(*map(bytes_dev, (*p, *q)), offsets=bytes_dev(off), out_dtype=dtype) for dtype in (BF16, F32)]
    a, b = ref.decode_columns(*p), ref.decode_columns(*q)
    for e in range(len(rooms)):
        check_exact([y[e] for y in ys], a[off[e]:off[e + 1]].T, b[off[e]:off[e + 1]].T)


def norm_error(y, want):
    return np.linalg.norm(f64(y) - want) / np.linalg.norm(want)


BOUND = {F32: 1e-6, BF16: 2.0**-9 + 1e-5}


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("rows,features", [(3, 304), (100, 260), (300, 272)])
@pytest.mark.parametrize("depth", [4480, 4608, 4736, 8191, 33000, 40000])
def test_error_of_normal_operands_against_the_norm(mx, direction, rows, features, depth):
    rng = np.random.default_rng(rows + depth)
    M, N, K = sizes(direction, rows, features, depth)
    normal = lambda *s: rng.standard_normal(s).astype(np.float32).astype(np.float64)  # noqa: E731
    if direction == "wgrad":
        p, q = ref.quant_columns(normal(M, N)), ref.quant_columns(normal(M, K))
        a, b = ref.decode_columns(*p).T, ref.decode_columns(*q).T
    else:
        p = ref.quant_rows(normal(M, K if direction == "fwd" else N))
        q = ref.e4m3_encode(normal(N, K) * 64), np.full((-(-N // 128), -(-K // 128)), 2.0**-6, np.float32)
        a, b = ref.decode_rows(*p), ref.decode_weight(*q)
        b = b if direction == "fwd" else b.T
    want = a @ b.T
    for dtype, bound in BOUND.items():
        assert norm_error(call(mx, direction)(*map(bytes_dev, (*p, *q)), out_dtype=dtype), want) < bound


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_error_of_an_experts_weight_gradient_against_its_norm(mx, dtype):
    rng = np.random.default_rng(51)
    rooms, N, K = [128, 4608, 0, 9216, 33024], 144, 272
    off = np.concatenate([[0], np.cumsum(rooms)]).astype(np.int32)
    normal = lambda n: rng.standard_normal((int(off[-1]), n)).astype(np.float32).astype(np.float64)  # noqa: E731
    p, q = ref.quant_columns(normal(N)), ref.quant_columns(normal(K))
    y = mx.fp8_matmul_wgrad(*map(bytes_dev, (*p, *q)), offsets=bytes_dev(off), out_dtype=dtype)
    a, b = ref.decode_columns(*p), ref.decode_columns(*q)
    for e, room in enumerate(rooms):
        if room:
            assert norm_error(y[e], a[off[e]:off[e + 1]].T @ b[off[e]:off[e + 1]]) < BOUND[dtype]
        else:
            assert not y[e].any()
