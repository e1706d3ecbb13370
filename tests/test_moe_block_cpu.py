"""Host-side checks of the norm, the router, the gated activation and the FP8
dispatch, without a GPU: the C entry points' refusals, the binding's, and the
64-bit references' gradients against differences."""

import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import moe_block_ref as bref

OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 4
FAKE = 0x10000000  # never dereferenced: every call below fails or returns before any launch


@pytest.fixture(scope="module")
def lib():
    return mxq.Library()


class _Norm(ctypes.Structure):
    """mxq_norm as include/mxq.h declares it."""
    _fields_ = [("dt", ctypes.c_int), ("weight_dt", ctypes.c_int), ("rows", ctypes.c_int64), ("K", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("y", ctypes.c_void_p), ("data", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class _NormGrad(ctypes.Structure):
    _fields_ = [("dt", ctypes.c_int), ("weight_dt", ctypes.c_int), ("rows", ctypes.c_int64), ("K", ctypes.c_int64), ("g", ctypes.c_void_p),
                ("ldg", ctypes.c_int64), ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("weight", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("g_h", ctypes.c_void_p), ("ldgh", ctypes.c_int64), ("d_h", ctypes.c_void_p), ("ldd", ctypes.c_int64), ("d_weight", ctypes.c_void_p)]


class _Route(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dt", ctypes.c_int), ("score", ctypes.c_int), ("tokens", ctypes.c_int64),
                ("experts", ctypes.c_int64), ("ld", ctypes.c_int64), ("topk", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("topk_groups", ctypes.c_int64), ("group_top", ctypes.c_int64), ("bias", ctypes.c_void_p), ("renormalize", ctypes.c_int),
                ("scale", ctypes.c_float)]


@pytest.mark.parametrize("cls,pack", [(_Norm, "_NORM"), (_NormGrad, "_NORM_GRAD"), (_Route, "_ROUTE")])
def test_the_binding_packs_the_structs(cls, pack):
    values = [i + 2 for i in range(len(cls._fields_))]
    packed = getattr(mxq, pack)(*values)
    assert len(packed) == ctypes.sizeof(cls)
    assert [getattr(cls.from_buffer_copy(packed), f) for f, _ in cls._fields_] == values


def norm(**kw):
    base = dict(rows=4, K=32, x=FAKE, ldx=32, weight=FAKE, eps=1e-6, data=FAKE, scales=FAKE)
    return bytes(_Norm(**(base | kw)))


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), UNSUPPORTED), (dict(weight_dt=2), UNSUPPORTED), (dict(dt=7), INVALID), (dict(rows=-1), INVALID), (dict(K=1 << 31, ldx=1 << 31), INVALID),
    (dict(ldx=31), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(residual=FAKE, ldr=31), INVALID),
    (dict(h=FAKE, ldh=32), INVALID), (dict(residual=FAKE, ldr=32, h=FAKE, ldh=31), INVALID), (dict(scales=None), INVALID), (dict(data=None), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(x=FAKE + 1), INVALID), (dict(weight=FAKE + 1), INVALID), (dict(y=FAKE + 1), INVALID),
    (dict(rstd=FAKE + 2), INVALID), (dict(residual=FAKE + 64, ldr=32, h=FAKE + 64, ldh=48), INVALID), (dict(residual=FAKE + 64, ldr=32, h=FAKE, ldh=48), INVALID),
    (dict(K=(1 << 30) + 1, ldx=1 << 31), INVALID), (dict(rows=0), OK), (dict(K=0, ldx=0), OK), (dict(data=None, scales=None), OK),
])
def test_norm_refusals(lib, change, status):
    assert lib.L.mxq_rmsnorm(norm(**change), None) == status


def norm_grad(**kw):
    base = dict(rows=4, K=32, g=FAKE, ldg=32, h=FAKE + 4096, ldh=32, weight=FAKE, rstd=FAKE, d_h=FAKE + 8192, ldd=32)
    return bytes(_NormGrad(**(base | kw)))


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), UNSUPPORTED), (dict(weight_dt=2), UNSUPPORTED), (dict(weight_dt=4), INVALID), (dict(rows=-1), INVALID), (dict(ldg=31), INVALID),
    (dict(ldh=31), INVALID), (dict(ldd=31), INVALID), (dict(g_h=FAKE, ldgh=31), INVALID), (dict(g=None), INVALID), (dict(h=None), INVALID),
    (dict(weight=None), INVALID), (dict(rstd=None), INVALID), (dict(d_h=None), INVALID), (dict(rstd=FAKE + 2), INVALID), (dict(g=FAKE + 1), INVALID),
    (dict(d_h=FAKE, ldd=48), INVALID), (dict(d_h=FAKE + 4096, ldd=48), INVALID), (dict(g_h=FAKE + 64, ldgh=32, d_h=FAKE + 64, ldd=48), INVALID),
    (dict(d_weight=FAKE), TOO_SMALL), (dict(d_weight=FAKE + 2), INVALID), (dict(rows=0), OK), (dict(K=0, ldg=0, ldh=0, ldd=0), OK),
])
def test_norm_grad_refusals(lib, change, status):
    assert lib.L.mxq_rmsnorm_grad(norm_grad(**change), None, 0, None) == status


def test_norm_grad_workspace(lib):
    assert lib.L.mxq_rmsnorm_grad_workspace(4, 32) == 4 * 32 * 4
    assert lib.L.mxq_rmsnorm_grad_workspace(8192, 7184) == 304 * 7184 * 4
    assert lib.L.mxq_rmsnorm_grad_workspace(0, 32) == lib.L.mxq_rmsnorm_grad_workspace(-1, 32) == 0
    assert lib.L.mxq_rmsnorm_grad(norm_grad(d_weight=FAKE), FAKE, 511, None) == TOO_SMALL
    assert lib.L.mxq_rmsnorm_grad(norm_grad(d_weight=FAKE), FAKE + 8, 512, None) == INVALID
    assert lib.L.mxq_rmsnorm_grad(None, None, 0, None) == INVALID


def route(**kw):
    base = dict(logits=FAKE, dt=1, tokens=4, experts=64, ld=64, topk=4, groups=1, topk_groups=1, group_top=1, renormalize=1, scale=1.0)
    return bytes(_Route(**(base | kw)))


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), UNSUPPORTED), (dict(dt=3), INVALID), (dict(score=2), INVALID), (dict(tokens=-1), INVALID), (dict(experts=0, ld=0), INVALID),
    (dict(experts=1025, ld=1025), INVALID), (dict(ld=63), INVALID), (dict(topk=0), INVALID), (dict(topk=33), INVALID),
    (dict(experts=3, ld=3), INVALID), (dict(tokens=1 << 30), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(logits=None), INVALID), (dict(logits=FAKE + 2), INVALID),
])
def test_route_refusals(lib, change, status):
    assert lib.L.mxq_moe_route(route(**change), FAKE, FAKE, None) == status
    assert lib.L.mxq_moe_route_grad(FAKE, route(**change), FAKE, FAKE, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(groups=0), INVALID), (dict(groups=64), INVALID), (dict(groups=5), INVALID), (dict(groups=4, topk_groups=5), INVALID), (dict(topk_groups=0), INVALID),
    (dict(group_top=0), INVALID), (dict(group_top=3), INVALID), (dict(experts=4, ld=4, topk=1, groups=4, group_top=2), INVALID),
    (dict(groups=32, topk_groups=1), INVALID), (dict(bias=FAKE + 2), INVALID), (dict(tokens=0, logits=None), OK),
])
def test_route_refusals_of_groups_and_bias(lib, change, status):
    assert lib.L.mxq_moe_route(route(**change), FAKE, FAKE, None) == status


def test_route_refuses_missing_outputs(lib):
    for ids, w in ((None, FAKE), (FAKE, None), (FAKE + 2, FAKE), (FAKE, FAKE + 1)):
        assert lib.L.mxq_moe_route(route(), ids, w, None) == INVALID
    assert lib.L.mxq_moe_route(None, FAKE, FAKE, None) == INVALID
    for g, ids, d in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (FAKE, FAKE, FAKE + 1)):
        assert lib.L.mxq_moe_route_grad(g, route(), ids, d, None) == INVALID


def test_gate_refusals(lib):
    L = lib.L
    assert L.mxq_silu_mul(FAKE, 2, 4, 32, 64, FAKE, None) == UNSUPPORTED
    assert L.mxq_silu_mul(FAKE, 5, 4, 32, 64, FAKE, None) == INVALID
    assert L.mxq_silu_mul(FAKE, 0, 4, 32, 63, FAKE, None) == INVALID  # ldx < 2H
    assert L.mxq_silu_mul(FAKE, 0, -4, 32, 64, FAKE, None) == INVALID
    assert L.mxq_silu_mul(FAKE, 0, 4, (1 << 29) + 1, 1 << 31, FAKE, None) == INVALID
    assert L.mxq_silu_mul(None, 0, 4, 32, 64, FAKE, None) == INVALID
    assert L.mxq_silu_mul(FAKE, 0, 4, 32, 64, None, None) == INVALID
    assert L.mxq_silu_mul(FAKE, 0, 4, 32, 64, FAKE + 1, None) == INVALID
    assert L.mxq_silu_mul(None, 0, 0, 32, 64, None, None) == OK
    for f in (L.mxq_fp8_silu_mul_1x128, L.mxq_fp8_silu_mul_128x1):
        assert f(FAKE, 2, 4, 32, 64, FAKE, FAKE, None) == UNSUPPORTED
        assert f(FAKE, 0, 4, 32, 64, None, FAKE, None) == INVALID
        assert f(FAKE, 0, 4, 32, 64, FAKE, None, None) == INVALID
        assert f(FAKE + 1, 0, 4, 32, 64, FAKE, FAKE, None) == INVALID
        assert f(None, 0, 4, 0, 0, None, None, None) == OK
    assert L.mxq_silu_mul_grad(FAKE, FAKE, 2, 4, 32, 32, 64, FAKE, None) == UNSUPPORTED
    assert L.mxq_silu_mul_grad(FAKE, FAKE, 0, 4, 32, 31, 64, FAKE, None) == INVALID
    assert L.mxq_silu_mul_grad(None, FAKE, 0, 4, 32, 32, 64, FAKE, None) == INVALID
    assert L.mxq_silu_mul_grad(FAKE, FAKE, 0, 4, 32, 32, 64, None, None) == INVALID


def test_dispatch_refusals(lib):
    f = lib.L.mxq_fp8_dispatch
    assert f(FAKE, FAKE, 4, 128, 127, FAKE, 2, 8, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 4, 128, 128, FAKE, 0, 8, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE, -1, 128, 128, FAKE, 2, 8, FAKE, FAKE, None) == INVALID
    assert f(None, FAKE, 4, 128, 128, FAKE, 2, 8, FAKE, FAKE, None) == INVALID
    assert f(FAKE, None, 4, 128, 128, FAKE, 2, 8, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 4, 128, 128, None, 2, 8, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 4, 128, 128, FAKE + 2, 2, 8, FAKE, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 4, 128, 128, FAKE, 2, 8, None, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 4, 128, 128, FAKE, 2, 8, FAKE, None, None) == INVALID
    assert f(None, None, 0, 128, 128, None, 2, 0, None, None, None) == OK


def test_the_binding_refuses_cpu_tensors(lib):
    x, w, u8 = torch.zeros(4, 128), torch.zeros(128), torch.zeros(4, 128, dtype=torch.uint8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: lib.rmsnorm(x, w), lambda: lib.rmsnorm_grad(x, x, w, torch.zeros(4)), lambda: lib.moe_route(x, 2),
              lambda: lib.moe_route_grad(torch.zeros(4, 2), x, ids), lambda: lib.silu_mul(x), lambda: lib.fp8_silu_mul_1x128(x),
              lambda: lib.fp8_silu_mul_128x1(x), lambda: lib.silu_mul_grad(x[:, :64], x), lambda: lib.fp8_dispatch(u8, u8[:, :1], ids.view(-1), 2)):
        with pytest.raises(ValueError):
            f()


# ------------------------------------------- the references' own gradients


def differences(f, x, at, step=1e-6):
    """d f / d x at the places `at`, by central differences."""
    out = []
    for i in at:
        a, b = x.copy(), x.copy()
        a.flat[i] += step
        b.flat[i] -= step
        out.append((f(a) - f(b)) / (2 * step))
    return np.array(out)


def test_norm_gradient_by_differences():
    rng = np.random.default_rng(0)
    h, w, g, g_h = rng.standard_normal((3, 20)), rng.standard_normal(20), rng.standard_normal((3, 20)), rng.standard_normal((3, 20))
    d, dw, _ = bref.norm_grad(g, h, w, bref.norm(h, w, 1e-3)[1], g_h)
    np.testing.assert_allclose(differences(lambda v: (g * bref.norm(v, w, 1e-3)[0]).sum() + (g_h * v).sum(), h, range(60)), d.ravel(), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(differences(lambda v: (g * bref.norm(h, v, 1e-3)[0]).sum(), w, range(20)), dw, rtol=1e-6, atol=1e-8)


def test_gate_gradient_by_differences():
    rng = np.random.default_rng(1)
    x, g = 2 * rng.standard_normal((3, 16)), rng.standard_normal((3, 8))
    np.testing.assert_allclose(differences(lambda v: (g * bref.gate(v)).sum(), x, range(48)), bref.gate_grad(g, x)[0].ravel(), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_by_differences(score, renormalize):
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((4, 9)), rng.standard_normal((4, 3))
    ids, _ = bref.route(x, 3, score=score)

    def loss(v):
        p = np.take_along_axis(bref.scores(v, score), ids, 1)
        return (g * 1.5 * (p / p.sum(1, keepdims=True) if renormalize else p)).sum()

    d, _ = bref.route_grad(g, x, ids, score, renormalize, 1.5)
    np.testing.assert_allclose(differences(loss, x, range(36)), d.ravel(), rtol=1e-6, atol=1e-8)


def test_the_reference_router_chooses_by_rank():
    x = np.array([[0.0, 3.0, 1.0, 3.0, -np.inf, 2.0]])
    ids, w = bref.route(x, 3, renormalize=True)
    assert ids.tolist() == [[1, 3, 5]]
    np.testing.assert_allclose(w, [[1, 1, np.exp(-1)]] / (2 + np.exp(-1)))
    ids, _ = bref.route(x, 2, groups=3, topk_groups=1, group_top=2)
    assert ids.tolist() == [[3, 2]]
    ids, w = bref.route(np.full((1, 4), -np.inf), 2)
    assert ids.tolist() == [[-1, -1]] and not w.any()
