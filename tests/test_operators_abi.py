"""Host-side validation of the routing and int8 calls: bad arguments are refused with the
documented status before any device work.  CPU only: nothing here launches a kernel."""

import ctypes
import os

import numpy as np
import pytest

import combine_topk_idx_expert_amd as ep
import plain_operators as plain
from combine_topk_idx_expert_amd._native import _RouteConfig

P = ctypes.c_void_p
S = ep.Status


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ep.lib_path()):
        import combine_topk_idx_expert_amd.build as b

        b.build()
    return ep.lib()


GOOD = dict(num_experts=256, num_topk=8, num_groups=8, topk_groups=4, score=1, group_score=1, renormalize=1, scale=2.5)


def route(L, cfg=None, type=0, logits=16, T=4, stride=256, bias=None, mask=None, idx=16, w=16):
    return L.ep_route(ctypes.byref(_RouteConfig(**{**GOOD, **(cfg or {})})), type, P(logits), T, stride, P(bias), P(mask),
                      P(idx), P(w), None)


def backward(L, cfg=None, type=0, logits=16, T=4, stride=256, idx=16, gw=16, grad=16):
    return L.ep_route_backward(ctypes.byref(_RouteConfig(**{**GOOD, **(cfg or {})})), type, P(logits), T, stride, P(idx),
                               P(gw), P(grad), None)


@pytest.mark.parametrize("change,status", [
    (dict(num_experts=0), S.ERR_SHAPE),
    (dict(num_experts=4104), S.ERR_SHAPE),
    (dict(num_topk=0), S.ERR_SHAPE),
    (dict(num_topk=33), S.ERR_SHAPE),
    (dict(num_groups=0), S.ERR_SHAPE),
    (dict(num_groups=7), S.ERR_SHAPE),
    (dict(num_groups=128), S.ERR_SHAPE),
    (dict(topk_groups=0), S.ERR_SHAPE),
    (dict(topk_groups=9), S.ERR_SHAPE),
    (dict(num_experts=16, topk_groups=3), S.ERR_SHAPE),  # 8 choices among 6 experts
    (dict(score=2), S.ERR_SHAPE),
    (dict(group_score=-1), S.ERR_SHAPE),
    (dict(scale=float("inf")), S.ERR_SHAPE),
    (dict(scale=float("nan")), S.ERR_SHAPE),
])
def test_route_config_is_checked(L, change, status):
    assert route(L, change) == status and L.ep_last_error()
    assert backward(L, change) == status


def test_route_arguments_are_checked(L):
    for call in (route, backward):
        assert call(L, type=3) == S.ERR_SHAPE
        assert call(L, T=-1) == S.ERR_SHAPE
        assert call(L, stride=255) == S.ERR_SHAPE
        assert call(L, T=(1 << 25) + 1) == S.ERR_OVERFLOW
        assert call(L, stride=1 << 41) == S.ERR_OVERFLOW
        assert call(L, logits=None) == S.ERR_NULL
        assert call(L, logits=2) == S.ERR_SHAPE
        assert call(L, idx=None) == S.ERR_NULL
        assert call(L, idx=4) == S.ERR_SHAPE
        assert call(L, T=0, logits=None, idx=None) == S.OK
    assert route(L, w=None) == S.ERR_NULL and route(L, w=2) == S.ERR_SHAPE and route(L, bias=2) == S.ERR_SHAPE
    assert backward(L, gw=None) == S.ERR_NULL and backward(L, grad=None) == S.ERR_NULL
    assert backward(L, grad=2) == S.ERR_SHAPE and backward(L, grad=1, type=1) == S.ERR_SHAPE
    assert L.ep_route(None, 0, None, 0, 0, None, None, None, None, None) == S.ERR_NULL


def quantize(L, type=0, x=16, rows=4, cols=64, stride=64, codes=16, scales=16):
    return L.ep_quantize_int8(type, P(x), rows, cols, stride, P(codes), P(scales), None)


def test_quantize_arguments_are_checked(L):
    assert quantize(L, type=-1) == S.ERR_SHAPE
    assert quantize(L, rows=-1) == S.ERR_SHAPE
    assert quantize(L, cols=0) == S.ERR_SHAPE
    assert quantize(L, stride=63) == S.ERR_SHAPE
    assert quantize(L, rows=(1 << 23) + 1) == S.ERR_OVERFLOW
    assert quantize(L, cols=(1 << 24) + 1, stride=1 << 25) == S.ERR_OVERFLOW
    assert quantize(L, x=None) == S.ERR_NULL and quantize(L, codes=None) == S.ERR_NULL
    assert quantize(L, scales=None) == S.ERR_NULL
    assert quantize(L, x=18) == S.ERR_SHAPE and quantize(L, scales=2) == S.ERR_SHAPE
    assert quantize(L, rows=0, x=None) == S.OK


def matmul(L, a=16, sa=16, M=4, w=16, sw=16, G=0, start=None, count=None, K=64, N=32, flags=0, type=1, out=16):
    return L.ep_matmul_int8(P(a), P(sa), M, P(w), P(sw), G, P(start), P(count), K, N, flags, type, P(out), None)


def test_matmul_arguments_are_checked(L):
    assert matmul(L, flags=2) == S.ERR_SHAPE
    assert matmul(L, type=5) == S.ERR_SHAPE
    assert matmul(L, M=-1) == S.ERR_SHAPE
    assert matmul(L, G=-1) == S.ERR_SHAPE
    assert matmul(L, G=4097, start=16, count=16) == S.ERR_SHAPE
    for K in (0, 8, 40, 131072):
        assert matmul(L, K=K) == S.ERR_SHAPE
    for N in (0, (1 << 20) + 2):
        assert matmul(L, N=N) == S.ERR_SHAPE
    assert matmul(L, N=33, flags=1) == S.ERR_SHAPE
    assert matmul(L, M=1 << 31) == S.ERR_OVERFLOW
    for name in ("a", "sa", "w", "sw", "out"):
        assert matmul(L, **{name: None}) == S.ERR_NULL
    assert matmul(L, G=2) == S.ERR_NULL and matmul(L, G=2, start=16) == S.ERR_NULL
    for name in ("a", "w", "out"):
        assert matmul(L, **{name: 8}) == S.ERR_SHAPE
    assert matmul(L, sa=2) == S.ERR_SHAPE and matmul(L, sw=2) == S.ERR_SHAPE
    assert matmul(L, G=2, start=4, count=16) == S.ERR_SHAPE and matmul(L, G=2, start=16, count=2) == S.ERR_SHAPE
    assert matmul(L, M=0, a=None) == S.OK


def test_expert_rows_needs_a_handle(L):
    assert L.ep_expert_rows(None, P(16), P(16), None) == S.ERR_NULL


def test_route_config_names_are_checked():
    with pytest.raises(ValueError):
        ep.RouteConfig(E=8, K=2, score="tanh")
    with pytest.raises(ValueError):
        ep.RouteConfig(E=8, K=2, group_score="mean")
    with pytest.raises(TypeError):
        ep.RouteConfig(E=8.5, K=2)
    assert ep.RouteConfig(E=8, K=2) == ep.RouteConfig(E=8, K=2, score="softmax")


def test_plain_route_hand_worked_rows():
    """The plain router on rows small enough to work by hand."""
    rc = ep.RouteConfig(E=4, K=2, score="sigmoid", num_groups=2, topk_groups=1, group_score="top2")
    x = np.array([[0.0, 0.0, 5.0, -9.0], [1.0, 1.0, 1.0, 1.0], [-np.inf, -np.inf, -np.inf, 2.0]])
    idx, w = plain.route(rc, x)
    # sums of two: 1.0 against 0.9933 + 0.0001; a tie; one choosable expert
    np.testing.assert_array_equal(idx, [[0, 1], [0, 1], [3, -1]])
    np.testing.assert_allclose(w, [[0.5, 0.5], [0.5, 0.5], [1.0, 0.0]])
    idx, _ = plain.route(ep.RouteConfig(E=4, K=2, num_groups=2, topk_groups=1), x)
    np.testing.assert_array_equal(idx, [[2, 3], [0, 1], [3, -1]])
    codes, scales = plain.quantize(np.array([[127.0, 0.5, 1.5, -2.5], [0.0, 0.0, 0.0, 0.0]]))
    np.testing.assert_array_equal(codes, [[127, 0, 2, -2], [0, 0, 0, 0]])
    np.testing.assert_array_equal(scales, np.float32([1.0, 0.0]))
