"""The gate's gradient where a projection was rounded to an infinity, and where the factors of a finite
gradient leave fp32 together: dg = d u s (1 + g (1 - s)), du = d g s.

One row at a time, with a one-hot row of a, so that column 0 of grad_w is the gradient of the projections.
"""

import numpy as np
import pytest
import torch

import combine_topk_idx_expert_amd as ep
import plain_expert_layer as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


def gate_gradient(g, u, d, dtype):
    """(dg, du) of one gate, up projection and gradient, each as the product's operand holds them."""
    pre = torch.tensor([g] * 8 + [u] * 8, device=DEV, dtype=dtype)[None]
    grad = torch.full((1, 8), d, device=DEV, dtype=dtype)
    one = torch.zeros(1, 8, device=DEV, dtype=dtype)
    one[0, 0] = 1.0
    w = torch.zeros(16, 8, device=DEV, dtype=dtype)
    _, gw = ep.matmul_backward(one, w, grad, gated=True, pre=pre, out=(None, torch.empty(16, 8, device=DEV)))
    got = gw[:, 0].cpu().double().numpy()
    assert np.array_equal(got[:8], np.full(8, got[0]), equal_nan=True) and np.array_equal(got[8:], np.full(8, got[8]), equal_nan=True)
    return got[0], got[8]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("u", [INF, -INF])
def test_infinite_up_projections(u, dtype):
    # a shut gate passes nothing, however large what it is multiplied with was
    for g in (-200.0, -5000.0, -INF):
        for d in (2.0, -0.5, 0.0):
            assert gate_gradient(g, u, d, dtype) == (0.0, 0.0), (g, d)
    # no gradient makes none
    for g in (-1.0, 0.0, 0.5, 2.5, 30.0, INF):
        assert gate_gradient(g, u, 0.0, dtype) == (0.0, 0.0), g
    # an open gate's is infinite, of the product's sign; its own slope turns at -1.28
    for g, sign in ((0.0, 1), (3.0, 1), (-1.0, 1), (-2.0, -1), (INF, 1)):
        dg, du = gate_gradient(g, u, 16.0, dtype)
        assert dg == sign * u, g
        assert np.isinf(du) == np.isinf(g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_stays_nan(dtype):
    assert np.isnan(gate_gradient(-200.0, NAN, 2.0, dtype)[0]) and gate_gradient(-200.0, NAN, 2.0, dtype)[1] == 0.0
    assert np.isnan(gate_gradient(NAN, INF, 2.0, dtype)).all()


@pytest.mark.parametrize("g", [-60.0, -87.0, -88.5, -90.0, -95.0, -200.0, 0.25, 40.0])
@pytest.mark.parametrize("d,u", [(1e25, 1e25), (-3e38, 2e38), (3.3e38, 3.3e38), (1e30, 1.0), (3e38, 0.25), (0.0, 3.3e38)])
def test_factors_that_leave_fp32_together(g, d, u):
    dtype = torch.bfloat16
    as_bf16 = lambda v: torch.tensor(v, dtype=dtype).double().item()
    g, d, u = as_bf16(g), as_bf16(d), as_bf16(u)
    got = gate_gradient(g, u, d, dtype)
    ref = plain.gate_backward(np.array([[g, u]]), np.array([[d]]))[0]
    # The sigmoid is off by 2^-17 of itself from its exponent's argument and some roundings, and by 2^-149 where it is
    # subnormal; so are the two products behind it, of slope (|g| + 1 times that) and with g.
    small = 2.0 ** -149
    own = np.array([abs(d * u) * (abs(g) + 3) * small, abs(d) * (abs(g) + 2) * small])
    tol = own + (2.0 ** -8 + 2.0 ** -15) * np.abs(ref) + 2.0 ** -134
    if g < -98:  # the sigmoid is below half of fp32's smallest value there
        tol = tol + np.abs(ref)
    largest = torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4)
    for value, want, t in zip(got, ref, tol):
        if np.isinf(value):
            assert abs(want) + t >= largest and np.sign(value) == np.sign(want)
        else:
            assert abs(value - want) <= t, (value, want, t)
