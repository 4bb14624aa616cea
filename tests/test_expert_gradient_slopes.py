"""Gradients of the gated 16-bit product against differences of the 64-bit function, along random directions.

Four roundings to fp16 stand between them, half a step u = 2^-11 of the value each (2^-25 below fp16's normal
range): of the projections, of the product's gradient d, and of the two results.  Each term's effect on the slope is
known, so as independent errors their deviation is at most u times the root of the sum of the squares; six of them
are allowed.  fp32 sums of up to 64 terms are far below that.
"""

import numpy as np
import pytest
import torch

import plain_expert_layer as plain

M, K, N = 40, 64, 48
U16, TINY16 = 2.0 ** -11, 2.0 ** -25


def f16(v):
    return np.asarray(v).astype(np.float16).astype(np.float64)


def problem():
    r = np.random.default_rng(1)
    x, v, c = f16(r.standard_normal((M, K))), f16(r.standard_normal((N, K)) / 4), f16(r.standard_normal((M, N // 2)))
    return x, v, c, [(r.standard_normal(x.shape), r.standard_normal(v.shape)) for _ in range(4)]


def slope_and_bound(x, v, c, e, h):
    """Slope along (e, h) by differences, and how far a right gradient's may be from it."""
    f = lambda x, v: (plain.gate(x @ v.T) * c).sum()
    step = 1e-5
    slope = (f(x + step * e, v + step * h) - f(x - step * e, v - step * h)) / (2 * step)
    pre, t = x @ v.T, e @ v.T + x @ h.T  # the projections, and how they move
    d = plain.gate_backward(pre, c)
    # what a projection's rounding does to d t: g and u of a column pair move both of its terms
    half = N // 2
    moved = np.empty_like(pre)
    for i, part in enumerate((slice(0, half), slice(half, N))):
        up, down = pre.copy(), pre.copy()
        up[:, part] += step
        down[:, part] -= step
        change = (plain.gate_backward(up, c) - plain.gate_backward(down, c)) / (2 * step) * t
        moved[:, part] = change[:, :half] + change[:, half:]
    off = lambda value, effect: ((np.maximum(U16 * np.abs(value), TINY16) * effect) ** 2).sum()
    variance = off(pre, moved) + off(d, t) + off(d @ v, e) + off(d.T @ x, h)
    return slope, 6 * variance ** 0.5


def test_a_weakened_slope_of_the_gate_shows():
    """The bound is small enough: without the term g (1 - s), or with the gate's two halves in each other's place, the
    slopes are outside of it."""
    x, v, c, directions = problem()
    pre = x @ v.T
    g, u = np.split(pre, 2, 1)
    s = 1 / (1 + np.exp(-g))
    right = plain.gate_backward(pre, c)
    weak = np.concatenate([c * u * s, c * g * s], 1)
    swapped = np.concatenate([right[:, N // 2:], right[:, :N // 2]], 1)
    few = right.copy()
    few[:, 3] *= 1.5  # one channel
    far = {"weak": 0, "swapped": 0, "few": 0}
    for e, h in directions:
        slope, bound = slope_and_bound(x, v, c, e, h)
        along = lambda d: ((d @ v) * e).sum() + ((d.T @ x) * h).sum()
        assert abs(along(right) - slope) < 1e-6 * (1 + abs(slope))
        for name, d in (("weak", weak), ("swapped", swapped), ("few", few)):
            far[name] += abs(along(d) - slope) > bound
    assert all(far.values()), far


@pytest.mark.gpu
def test_gradients_agree_with_differences():
    import combine_topk_idx_expert_amd as ep

    x, v, c, directions = problem()
    a, w, grad = (torch.from_numpy(t).to("cuda:0", torch.float16) for t in (x, v, c))
    pre = torch.empty(M, N, dtype=torch.float16, device="cuda:0")
    ep.matmul(a, w, gated=True, pre=pre)
    ga, gw = (t.cpu().double().numpy() for t in ep.matmul_backward(a, w, grad, gated=True, pre=pre))
    for e, h in directions:
        slope, bound = slope_and_bound(x, v, c, e, h)
        got = (ga * e).sum() + (gw * h).sum()
        print("[slopes]", slope, got - slope, bound, flush=True)
        assert abs(got - slope) < bound
