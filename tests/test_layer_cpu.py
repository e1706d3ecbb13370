"""Host-side checks of the FP8 linear layer and the mixture-of-experts entry
points, without a GPU: the C entry points' refusals, and the binding's."""

import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import layer_ref as ref

OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 4
FAKE = 0x10000000  # never dereferenced: every call below fails or returns before any launch


@pytest.fixture(scope="module")
def lib():
    return mxq.Library()


class _Product(ctypes.Structure):
    """mxq_fp8_product as include/mxq.h declares it."""
    _fields_ = [("dir", ctypes.c_int), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("a", ctypes.c_void_p), ("lda", ctypes.c_int64), ("a_scales", ctypes.c_void_p),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("b_scales", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_dt", ctypes.c_int), ("ldo", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("E", ctypes.c_int64)]


def product(**kw):
    base = dict(dir=0, M=4, N=256, K=128, a=FAKE, lda=128, a_scales=FAKE, b=FAKE, ldb=128, b_scales=FAKE, out=FAKE,
                out_dt=0, ldo=256, offsets=None, E=0)
    return bytes(_Product(**(base | kw)))


def test_the_binding_packs_the_struct():
    values = (2, 3, 5, 7, 11, 13, 17, 19, 23, 29, 31, 1, 37, 41, 43)
    p = _Product(*values)
    packed = mxq._PRODUCT(*values)
    assert len(packed) == ctypes.sizeof(p)
    assert tuple(getattr(_Product.from_buffer_copy(packed), f) for f, _ in _Product._fields_) == values


@pytest.mark.parametrize("change,status", [
    (dict(dir=3), INVALID), (dict(M=-1), INVALID), (dict(K=(1 << 30) + 1, lda=1 << 31, ldb=1 << 31), INVALID),
    (dict(out_dt=2), UNSUPPORTED), (dict(out_dt=5), INVALID), (dict(lda=127), INVALID), (dict(ldb=64), INVALID),
    (dict(ldo=255), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(a_scales=None), INVALID),
    (dict(b_scales=None), INVALID), (dict(b_scales=FAKE + 2), INVALID), (dict(out=None), INVALID),
    (dict(out=FAKE + 1), INVALID), (dict(offsets=FAKE, E=0), INVALID), (dict(offsets=FAKE, E=1025), INVALID),
    (dict(offsets=FAKE + 2, E=2), INVALID), (dict(a=FAKE + 1), TOO_SMALL), (dict(lda=130), TOO_SMALL),
    (dict(M=0), OK), (dict(N=0), OK), (dict(dir=1, lda=255), INVALID), (dict(dir=2, lda=256, ldo=127), INVALID),
])
def test_product_refusals(lib, change, status):
    assert lib.L.mxq_fp8_matmul(product(**change), None, 0, None) == status


def test_product_refuses_no_description(lib):
    assert lib.L.mxq_fp8_matmul(None, None, 0, None) == INVALID
    assert lib.L.mxq_fp8_matmul_workspace(None) == 0


def test_workspace_of_rows_that_are_not_aligned(lib):
    need = lambda **kw: lib.L.mxq_fp8_matmul_workspace(product(**kw))  # noqa: E731
    assert need() == 0
    assert need(K=100, lda=100, ldb=100) == 4 * 112 + 256 * 112
    assert need(K=100, lda=112, ldb=112) == 0
    assert need(M=1, K=100, lda=100, ldb=112) == 0  # one row has no stride
    assert need(a=FAKE + 8) == 4 * 128
    assert need(K=100, lda=112, ldb=100, offsets=FAKE, E=3) == 3 * 256 * 112
    assert lib.L.mxq_fp8_matmul(product(a=FAKE + 8), FAKE, 511, None) == TOO_SMALL
    assert lib.L.mxq_fp8_matmul(product(a=FAKE + 8), FAKE + 4, 512, None) == INVALID


def test_quant_refusals(lib):
    for f in (lib.L.mxq_fp8_quant_1x128, lib.L.mxq_fp8_quant_128x1):
        assert f(FAKE, 2, 4, 32, 32, None, 1, 4, FAKE, FAKE, None) == UNSUPPORTED
        assert f(FAKE, 9, 4, 32, 32, None, 1, 4, FAKE, FAKE, None) == INVALID
        assert f(FAKE, 0, 4, 32, 31, None, 1, 4, FAKE, FAKE, None) == INVALID   # ld < K
        assert f(FAKE, 0, 4, 32, 32, None, 1, 5, FAKE, FAKE, None) == INVALID   # rows without an index
        assert f(FAKE, 0, 4, 32, 32, FAKE, 0, 5, FAKE, FAKE, None) == INVALID   # divisor
        assert f(FAKE, 0, 4, 32, 32, FAKE + 1, 1, 5, FAKE, FAKE, None) == INVALID
        assert f(FAKE + 1, 0, 4, 32, 32, None, 1, 4, FAKE, FAKE, None) == INVALID
        assert f(None, 0, 4, 32, 32, None, 1, 4, FAKE, FAKE, None) == INVALID
        assert f(FAKE, 0, 4, 32, 32, None, 1, 4, None, FAKE, None) == INVALID
        assert f(None, 0, 0, 32, 32, None, 1, 0, None, None, None) == OK


def test_sort_refusals_and_sizes(lib):
    f = lib.L.mxq_moe_sort
    assert f(FAKE, 4, 2, 0, 1, FAKE, FAKE, FAKE, None, 0, None) == INVALID
    assert f(FAKE, 4, 2, 2049, 1, FAKE, FAKE, FAKE, None, 0, None) == INVALID
    assert f(FAKE, 4, 2, 8, 0, FAKE, FAKE, FAKE, None, 0, None) == INVALID
    assert f(FAKE, 1 << 30, 2, 8, 1, FAKE, FAKE, FAKE, None, 0, None) == INVALID
    assert f(FAKE, 1 << 20, 2, 2048, 1 << 20, FAKE, FAKE, FAKE, None, 0, None) == INVALID  # capacity
    assert f(None, 4, 2, 8, 1, FAKE, FAKE, FAKE, None, 0, None) == INVALID
    assert f(FAKE, 4, 2, 8, 1, None, FAKE, FAKE, None, 0, None) == INVALID
    assert f(FAKE, 4, 2, 8, 1, FAKE + 2, FAKE, FAKE, None, 0, None) == INVALID
    assert f(FAKE, 1 << 20, 2, 8, 1, FAKE, FAKE, FAKE, None, 0, None) == TOO_SMALL
    assert lib.L.mxq_moe_capacity(48, 2, 32, 1) == 96
    assert lib.L.mxq_moe_capacity(3, 2, 32, 128) == 6 + 6 * 127
    assert lib.L.mxq_moe_capacity(0, 2, 32, 128) == 0


def test_rows_refusals(lib):
    L = lib.L
    assert L.mxq_moe_dispatch(FAKE, 2, 4, 8, 8, FAKE, 2, 8, FAKE, None) == UNSUPPORTED
    assert L.mxq_moe_dispatch(FAKE, 0, 4, 8, 7, FAKE, 2, 8, FAKE, None) == INVALID
    assert L.mxq_moe_dispatch(FAKE, 0, 4, 8, 8, FAKE, 0, 8, FAKE, None) == INVALID
    assert L.mxq_moe_dispatch(FAKE, 0, 4, 8, 8, None, 2, 8, FAKE, None) == INVALID
    assert L.mxq_moe_dispatch(None, 0, 4, 8, 8, None, 2, 0, None, None) == OK
    assert L.mxq_moe_combine(FAKE, 2, 4, 8, 8, FAKE, None, 2, 2, FAKE, None) == UNSUPPORTED
    assert L.mxq_moe_combine(FAKE, 0, 4, 8, 8, None, None, 2, 2, FAKE, None) == INVALID
    assert L.mxq_moe_combine(FAKE, 1, 4, 8, 8, FAKE, FAKE + 2, 2, 2, FAKE, None) == INVALID
    assert L.mxq_moe_combine(None, 0, 0, 8, 8, None, None, 0, 2, None, None) == OK
    assert L.mxq_moe_combine_grad(FAKE, FAKE, 2, 2, 2, 4, 8, 8, 8, FAKE, FAKE, FAKE, FAKE, FAKE, None) == UNSUPPORTED
    assert L.mxq_moe_combine_grad(FAKE, FAKE, 0, 2, 2, 4, 8, 8, 8, FAKE, FAKE, None, FAKE, FAKE, None) == INVALID
    assert L.mxq_moe_combine_grad(FAKE, FAKE, 0, 2, 2, 4, 8, 8, 8, None, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert L.mxq_moe_combine_grad(FAKE, FAKE, 0, 2, 2, 4, 8, 7, 8, FAKE, FAKE, FAKE, FAKE, FAKE, None) == INVALID


def test_the_binding_refuses_cpu_tensors(lib):
    x, u8 = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.uint8)
    for f in (lambda: lib.fp8_quant_1x128(x), lambda: lib.fp8_quant_128x1(x),
              lambda: lib.fp8_matmul(u8, u8[:, :1].contiguous(), u8, torch.ones(1, 1)),
              lambda: lib.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 3),
              lambda: lib.moe_dispatch(x, torch.zeros(4, dtype=torch.int32), 1),
              lambda: lib.moe_combine(x, torch.zeros(4, 1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            f()


def test_the_binding_sees_rows():
    t = torch.zeros(6, 8, 32, dtype=torch.uint8)
    assert mxq._matrix(t, "t") == (48, 32, 32)
    assert mxq._matrix(t[:, :, :20], "t") == (48, 20, 32)
    assert mxq._matrix(t[0, 0], "t") == (1, 32, 32)
    assert mxq._matrix(t[0, :1, 3:9], "t") == (1, 6, 6)
    assert mxq._matrix(t[0, :, :1], "t") == (8, 1, 32)
    assert mxq._matrix(t[:0], "t") == (0, 32, 32)
    assert mxq._matrix(t[0, :, :0], "t") == (8, 0, 0)
    for bad in (t[0, :1].expand(8, 32), t[0].t(), t[:, :4], t[0, :, ::2], torch.zeros(())):
        with pytest.raises(ValueError):
            mxq._matrix(bad, "t")
    with pytest.raises(ValueError):
        mxq._matrix(t, "t", 2)


def test_the_reference_rounds_to_nearest_even():
    assert ref.e4m3_encode(np.array([448.0, 0.0, -0.0, 2.0**-10, 3 * 2.0**-10, 17.0, 19.0, -1.0])).tolist() == [
        0x7E, 0, 0x80, 0, 2, 0x58, 0x5A, 0xB8]
    back = ref.e4m3_decode(np.arange(127, dtype=np.uint8))
    np.testing.assert_array_equal(ref.e4m3_encode(back), np.arange(127))
    torch_cast = torch.from_numpy(np.linspace(-448, 448, 20001, dtype=np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.e4m3_encode(np.linspace(-448, 448, 20001, dtype=np.float32).astype(np.float64)), torch_cast)
