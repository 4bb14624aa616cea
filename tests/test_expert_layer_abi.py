"""Host-side validation of the norm, E4M3 and 16-bit product calls: bad arguments are refused with
the documented status before any device work.  CPU only: nothing here launches a kernel."""

import ctypes
import os

import numpy as np
import pytest

import combine_topk_idx_expert_amd as ep
import plain_expert_layer as plain

P = ctypes.c_void_p
S = ep.Status


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ep.lib_path()):
        import combine_topk_idx_expert_amd.build as b

        b.build()
    return ep.lib()


def quantize(L, type=0, x=16, rows=4, cols=64, stride=64, flags=0, codes=16, scales=16):
    return L.ep_quantize_fp8(type, P(x), rows, cols, stride, flags, P(codes), P(scales), None)


def test_quantize_arguments_are_checked(L):
    assert quantize(L, type=3) == S.ERR_SHAPE and L.ep_last_error()
    assert quantize(L, flags=1) == S.ERR_SHAPE
    assert quantize(L, rows=-1) == S.ERR_SHAPE
    assert quantize(L, cols=0) == S.ERR_SHAPE
    assert quantize(L, stride=63) == S.ERR_SHAPE
    assert quantize(L, rows=(1 << 23) + 1) == S.ERR_OVERFLOW
    assert quantize(L, cols=(1 << 24) + 1, stride=1 << 25) == S.ERR_OVERFLOW
    assert quantize(L, stride=1 << 41) == S.ERR_OVERFLOW
    assert quantize(L, rows=1 << 23, cols=1 << 15, stride=1 << 15) == S.ERR_OVERFLOW  # 2^31 scales
    for name in ("x", "codes", "scales"):
        assert quantize(L, **{name: None}) == S.ERR_NULL
    assert quantize(L, x=18) == S.ERR_SHAPE and quantize(L, x=17, type=1) == S.ERR_SHAPE
    assert quantize(L, scales=2) == S.ERR_SHAPE
    assert quantize(L, rows=0, x=None) == S.OK


def norm(L, type=1, x=16, xs=64, res=None, rs=64, w=16, wt=1, eps=1e-6, rows=4, cols=64, total=None, y=16, codes=None,
         scales=None):
    return L.ep_rms_norm(type, P(x), xs, P(res), rs, P(w), wt, eps, rows, cols, P(total), P(y), P(codes), P(scales), None)


def test_norm_arguments_are_checked(L):
    assert norm(L, type=-1) == S.ERR_SHAPE
    assert norm(L, wt=2) == S.ERR_SHAPE and norm(L, type=0, wt=1) == S.ERR_SHAPE
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert norm(L, eps=eps) == S.ERR_SHAPE
    assert norm(L, rows=-1) == S.ERR_SHAPE and norm(L, cols=0) == S.ERR_SHAPE
    assert norm(L, rows=(1 << 23) + 1) == S.ERR_OVERFLOW
    assert norm(L, cols=32769, xs=40000) == S.ERR_OVERFLOW
    assert norm(L, xs=63) == S.ERR_SHAPE and norm(L, xs=1 << 41) == S.ERR_OVERFLOW
    assert norm(L, x=None) == S.ERR_NULL and norm(L, w=None) == S.ERR_NULL
    assert norm(L, y=None) == S.ERR_NULL  # nothing to write
    assert norm(L, codes=16) == S.ERR_NULL  # no scales
    assert norm(L, res=16) == S.ERR_NULL  # no total
    assert norm(L, res=16, total=16, rs=63) == S.ERR_SHAPE
    for name in ("x", "w", "y"):
        assert norm(L, **{name: 17}) == S.ERR_SHAPE
    assert norm(L, w=18, wt=0) == S.ERR_SHAPE
    assert norm(L, res=17, total=16) == S.ERR_SHAPE and norm(L, res=16, total=17) == S.ERR_SHAPE
    assert norm(L, codes=16, scales=2) == S.ERR_SHAPE
    assert norm(L, rows=0, x=None) == S.OK


def norm_back(L, type=1, x=16, xs=64, w=16, wt=1, eps=1e-6, g=16, gs=64, t=None, ts=64, rows=4, cols=64, gx=16, gw=16,
              space=16):
    return L.ep_rms_norm_backward(type, P(x), xs, P(w), wt, eps, P(g), gs, P(t), ts, rows, cols, P(gx), P(gw), P(space), None)


def test_norm_backward_arguments_are_checked(L):
    assert norm_back(L, type=4) == S.ERR_SHAPE and norm_back(L, wt=2) == S.ERR_SHAPE
    assert norm_back(L, eps=0.0) == S.ERR_SHAPE
    assert norm_back(L, rows=-1) == S.ERR_SHAPE and norm_back(L, cols=0) == S.ERR_SHAPE
    assert norm_back(L, cols=32769) == S.ERR_OVERFLOW
    for name in ("xs", "gs"):
        assert norm_back(L, **{name: 63}) == S.ERR_SHAPE
    assert norm_back(L, t=16, ts=63) == S.ERR_SHAPE
    for name in ("x", "w", "g", "gx", "gw", "space"):
        assert norm_back(L, **{name: None}) == S.ERR_NULL
    for name in ("x", "w", "g", "gx"):
        assert norm_back(L, **{name: 17}) == S.ERR_SHAPE
    assert norm_back(L, gw=2) == S.ERR_SHAPE and norm_back(L, space=2) == S.ERR_SHAPE and norm_back(L, t=17) == S.ERR_SHAPE
    n = ctypes.c_int64(-1)
    assert L.ep_rms_norm_backward_workspace(1, 100, 4096, None) == S.ERR_NULL
    assert L.ep_rms_norm_backward_workspace(7, 100, 4096, ctypes.byref(n)) == S.ERR_SHAPE
    for rows in (0, 1, 1000, 1 << 23):
        assert L.ep_rms_norm_backward_workspace(1, rows, 4096, ctypes.byref(n)) == S.OK
        assert 0 <= n.value <= (rows and 2560 * 4096 * 4) and n.value % (4096 * 4) == 0


def fp8(L, a=16, sa=16, M=4, w=16, sw=16, G=0, start=None, count=None, K=64, N=32, flags=0, type=1, out=16):
    return L.ep_matmul_fp8(P(a), P(sa), M, P(w), P(sw), G, P(start), P(count), K, N, flags, type, P(out), None)


def test_matmul_fp8_arguments_are_checked(L):
    assert fp8(L, flags=4) == S.ERR_SHAPE and fp8(L, type=5) == S.ERR_SHAPE
    assert fp8(L, M=-1) == S.ERR_SHAPE and fp8(L, G=-1) == S.ERR_SHAPE
    assert fp8(L, G=4097, start=16, count=16) == S.ERR_SHAPE
    for K in (0, 8, 40, 131072):
        assert fp8(L, K=K) == S.ERR_SHAPE
    for N in (0, (1 << 20) + 2):
        assert fp8(L, N=N) == S.ERR_SHAPE
    assert fp8(L, N=33, flags=1) == S.ERR_SHAPE
    assert fp8(L, M=1 << 31) == S.ERR_OVERFLOW
    for name in ("a", "sa", "w", "sw", "out"):
        assert fp8(L, **{name: None}) == S.ERR_NULL
    assert fp8(L, G=2) == S.ERR_NULL and fp8(L, G=2, start=16) == S.ERR_NULL
    for name in ("a", "w", "out"):
        assert fp8(L, **{name: 8}) == S.ERR_SHAPE
    assert fp8(L, sa=2) == S.ERR_SHAPE and fp8(L, sw=2) == S.ERR_SHAPE
    assert fp8(L, G=2, start=4, count=16) == S.ERR_SHAPE and fp8(L, G=2, start=16, count=2) == S.ERR_SHAPE
    assert fp8(L, M=0, a=None) == S.OK and fp8(L, M=0, flags=3) == S.OK


def half(L, type=1, a=16, M=4, w=16, G=0, start=None, count=None, K=64, N=32, flags=0, pre=None, out=16):
    return L.ep_matmul(type, P(a), M, P(w), G, P(start), P(count), K, N, flags, P(pre), P(out), None)


def test_matmul_arguments_are_checked(L):
    assert half(L, type=0) == S.ERR_SHAPE and half(L, type=3) == S.ERR_SHAPE
    assert half(L, flags=2) == S.ERR_SHAPE
    for K in (0, 4, 12, 131064):
        assert half(L, K=K) == S.ERR_SHAPE
    assert half(L, N=0) == S.ERR_SHAPE and half(L, N=33, flags=1) == S.ERR_SHAPE
    assert half(L, M=1 << 31) == S.ERR_OVERFLOW
    assert half(L, pre=16) == S.ERR_SHAPE  # not gated
    for name in ("a", "w", "out"):
        assert half(L, **{name: None}) == S.ERR_NULL and half(L, **{name: 8}) == S.ERR_SHAPE
    assert half(L, flags=1, pre=8) == S.ERR_SHAPE
    assert half(L, G=2, start=16) == S.ERR_NULL and half(L, G=2, start=4, count=16) == S.ERR_SHAPE
    assert half(L, M=0, a=None) == S.OK


def back(L, type=1, a=16, M=4, w=16, grad=16, pre=None, G=0, start=None, count=None, K=64, N=32, flags=0, ga=16, gw=16,
         gtype=1, space=16):
    return L.ep_matmul_backward(type, P(a), M, P(w), P(grad), P(pre), G, P(start), P(count), K, N, flags, P(ga), P(gw), gtype,
                                P(space), None)


def test_matmul_backward_arguments_are_checked(L):
    assert back(L, type=0) == S.ERR_SHAPE and back(L, gtype=2) == S.ERR_SHAPE and back(L, flags=8) == S.ERR_SHAPE
    assert back(L, K=12) == S.ERR_SHAPE and back(L, N=36) == S.ERR_SHAPE
    assert back(L, N=40, flags=1, pre=16) == S.ERR_SHAPE
    assert back(L, ga=None, gw=None) == S.ERR_NULL
    for name in ("a", "w", "grad"):
        assert back(L, **{name: None}) == S.ERR_NULL and back(L, **{name: 8}) == S.ERR_SHAPE
    for name in ("ga", "gw", "space"):
        assert back(L, **{name: 8}) == S.ERR_SHAPE
    assert back(L, flags=1) == S.ERR_NULL and back(L, pre=16) == S.ERR_SHAPE
    assert back(L, flags=1, pre=16, space=None) == S.ERR_NULL
    assert back(L, G=2, start=16) == S.ERR_NULL and back(L, G=2, start=4, count=16) == S.ERR_SHAPE


@pytest.mark.parametrize("M,G,K,N,gated", [(0, 0, 64, 64, False), (1, 0, 4096, 4096, True), (32768, 0, 512, 512, False),
                                           (65536, 32, 4096, 4096, True), (100, 4096, 8, 16, True),
                                           ((1 << 31) - 1, 0, 8, 8, False)])
def test_matmul_backward_workspace_holds_the_gate_and_the_slices(L, M, G, K, N, gated):
    n = ctypes.c_int64(-1)
    assert L.ep_matmul_backward_workspace(M, G, K, N, int(gated), ctypes.byref(n)) == S.OK
    assert n.value >= (M * N * 2 if gated else 0)
    # slices are for fewer than half the 256 CUs' tiles of 128 x 256, so they stay small
    assert n.value <= (M * N * 2 + 256 if gated else 0) + 256 * 128 * 256 * 4 * 2
    assert L.ep_matmul_backward_workspace(M, G, K, N, int(gated), None) == S.ERR_NULL
    assert L.ep_matmul_backward_workspace(M, G, K, N + 1, int(gated), ctypes.byref(n)) == S.ERR_SHAPE


def test_plain_gate_gradient_agrees_with_differences():
    r = np.random.default_rng(1)
    pre, d = r.standard_normal((5, 12)) * 4, r.standard_normal((5, 6))
    got = plain.gate_backward(pre, d)
    for i in range(5):
        for j in range(12):
            step = np.zeros_like(pre)
            step[i, j] = 1e-6
            slope = ((plain.gate(pre + step) - plain.gate(pre - step)) * d).sum() / 2e-6
            assert abs(slope - got[i, j]) < 1e-7 * (1 + abs(slope))


def test_plain_e4m3_codes():
    v = plain.E4M3
    assert v[0x7E] == 448 and v[0x38] == 1 and v[0x01] == 2.0 ** -9 and np.isnan(v[0x7F])
    finite = np.array([c for c in range(256) if c & 127 != 127])
    np.testing.assert_array_equal(plain.encode(v[finite]), finite)
    # ties go to the even code
    assert plain.encode(np.array([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [0x38, 0x3A, 0x00, 0x02]
