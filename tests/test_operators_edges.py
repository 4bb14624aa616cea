"""Routing and int8 operators at the borders of their number ranges, against plain 64-bit
implementations: group sums beyond fp32, ties under a bias, rows without a choosable logit, NaN
in the gradient, gates that close.

Tolerances come from the number of roundings; u is half a step of fp32, 2^-24.
"""

import numpy as np
import pytest
import torch

import combine_topk_idx_expert_amd as ep
import plain_operators as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
LOWEST = torch.finfo(torch.float32).min
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def check_ids(rc, x, bias):
    idx, w = ep.route(rc, x, bias=bias)
    ref_idx, ref_w = plain.route(rc, f64(x), None if bias is None else f64(bias))
    np.testing.assert_array_equal(idx.cpu().numpy(), ref_idx)
    # the exponential's argument is off by a few u for each unit of its size, the rest by a few u
    top = np.abs(np.where(np.isfinite(f64(x)), f64(x), 0)).max()
    np.testing.assert_allclose(f64(w), ref_w, rtol=(40 + rc.K + 8 * min(top, 110)) * U, atol=2.0 ** -125)
    return idx


# -------------------------------------------------------------------------------- routing

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,groups,kept", [(16, 6, 4, 2), (32, 10, 4, 2), (64, 8, 8, 2), (256, 8, 8, 4), (200, 12, 8, 4),
                                             (512, 16, 8, 2), (320, 10, 64, 7), (128, 12, 16, 5),
                                             (64, 10, 8, 2), (64, 8, 8, 1), (200, 12, 8, 1), (512, 16, 8, 1),
                                             (320, 11, 64, 3), (4096, 32, 64, 1)])
def test_route_groups_whose_sum_leaves_fp32(score, E, K, groups, kept):
    """Experts switched off by a bias of the lowest fp32 value: the sum of two such keys lies below fp32, and
    a group of them still comes before a group without a choosable expert."""
    g = generator(E + K)
    size = E // groups
    rc = ep.RouteConfig(E=E, K=K, score=score, num_groups=groups, topk_groups=kept, group_score="top2")
    x = torch.randn(40, E, generator=g, device=DEV)
    live = kept - 1                                   # groups that are left as they are, at the end
    x[:, :size] = -INF                                # the first group has no choosable expert
    x[20:, size:2 * size] = -INF                      # nor has the second, in half of the rows
    off = torch.randn(E, generator=g, device=DEV) * 0.01
    for low in (LOWEST, -2.0e38, -1.0e38):
        bias = off.clone()
        bias[size:E - live * size] = low
        check_ids(rc, x, bias)
        if groups - live >= 4:                        # groups switched off by different amounts
            bias[2 * size:3 * size] = 0.75 * low
            check_ids(rc, x, bias)
    for high in (3.0e38, torch.finfo(torch.float32).max):  # and sums above fp32
        bias = off.clone()
        bias[size:2 * size] = high
        bias[E - size:] = 0.9 * high
        check_ids(rc, x, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,groups,kept,group_score", [
    (61, 8, 1, 1, "max"), (62, 8, 1, 1, "max"), (63, 16, 1, 1, "max"), (250, 8, 1, 1, "max"), (253, 13, 1, 1, "max"),
    (255, 8, 3, 2, "top2"), (54, 11, 6, 3, "top2"), (500, 9, 1, 1, "max"), (497, 8, 7, 3, "max")])
def test_route_ties_under_a_bias_at_the_end_of_a_row(score, E, K, groups, kept, group_score):
    """Few logits, few biases that are no sums of powers of two: keys of equal parts tie, wherever the
    bias was read."""
    g = generator(E)
    rc = ep.RouteConfig(E=E, K=K, score=score, num_groups=groups, topk_groups=kept, group_score=group_score)
    store = torch.empty(E + 4, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randint(-2, 3, (300, E), generator=g, device=DEV).to(dtype)
        x[0] = 0.0
        x[1, : E - 3] = -1.0
        x[2, ::2] = -INF
        for values in ([0.1], [0.3, 0.7], [-0.3, 0.1, 1.1]):
            v = torch.tensor(values, device=DEV)
            b = v[torch.randint(0, len(values), (E,), generator=g, device=DEV)]
            for off in (0, 1):                        # a bias that is not 16-byte aligned
                bias = store[off:off + E]
                bias.copy_(b)
                check_ids(rc, x, bias)


# ------------------------------------------------------------------- gradient of the router

GRADIENTS = [(64, 4), (61, 5), (256, 8), (600, 6), (256, 12), (256, 20), (1030, 5)]


def gradient_tolerance(x, K, scale, g, ref, dtype):
    top = np.abs(np.where(np.isfinite(x), x, 0)).max()
    big = np.abs(g).max(1, keepdims=True)
    return ((40 + 8 * min(top, 110) + 5 * K) * U * scale * 2 * big + half_step(dtype) * np.abs(ref)
            + (2.0 ** -25 if dtype == torch.float16 else 0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,K", GRADIENTS)
def test_route_backward_of_rows_without_a_score(score, renorm, E, K):
    """Ids that name logits of -Inf, in rows of nothing else and in ordinary ones: their scores are 0, and
    nothing reaches them."""
    g = generator(E * K)
    for dtype in DTYPES.values():
        x = torch.randn(9, E, generator=g, device=DEV).to(dtype)
        idx = torch.rand(9, E, generator=g, device=DEV).argsort(1)[:, :K].contiguous()
        gw = torch.randn(9, K, generator=g, device=DEV)
        x[0] = -INF
        x[1] = -INF
        x[1, idx[1, 0]] = 0.5                         # one of the choices alone
        x[2] = -INF
        x[2, (set(range(E)) - set(idx[2].tolist())).pop()] = 0.5  # an expert that was not chosen
        x[3].scatter_(0, idx[3], -INF)                # every choice
        x[4, idx[4, K - 1]] = -INF
        x[5] = torch.finfo(dtype).min
        rc = ep.RouteConfig(E=E, K=K, score=score, renormalize=renorm, scale=2.5)
        got = f64(ep.route_backward(rc, x, idx, gw))
        ref = plain.route_backward(rc, f64(x), idx.cpu().numpy(), f64(gw))
        ref[0] = 0.0
        assert np.isfinite(got).all()
        xs = np.where(np.abs(f64(x)) < 1e3, f64(x), 0)
        tol = gradient_tolerance(xs, K, 2.5, f64(gw), ref, dtype)
        assert (np.abs(got - ref) <= tol).all(), (dtype, np.abs(got - ref).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,K", GRADIENTS)
def test_route_backward_shows_nan(score, renorm, E, K):
    """A NaN logit makes NaN of what it reaches: the whole row where the softmax runs over it, the token's
    choices where it is one of them and they are renormalised, itself alone otherwise."""
    g = generator(E + K)
    nan = float("nan")
    for dtype in DTYPES.values():
        x = torch.randn(8, E, generator=g, device=DEV).to(dtype)
        idx = torch.rand(8, E, generator=g, device=DEV).argsort(1)[:, :K].contiguous()
        gw = torch.randn(8, K, generator=g, device=DEV)
        x[1, idx[1, 0]] = nan                         # a choice
        x[2, idx[2, K - 1]] = nan
        x[2, idx[2, 0]] = -INF                        # beside one of score 0
        other = (set(range(E)) - set(idx[3].tolist())).pop()
        x[3, other] = nan                             # no choice
        x[4] = nan
        x[5] = nan
        idx[5] = -1                                   # a token that was not routed
        idx[6, K - 1] = -1                            # an unused slot
        x[6, idx[6, 0]] = nan
        rc = ep.RouteConfig(E=E, K=K, score=score, renormalize=renorm)
        dx = ep.route_backward(rc, x, idx, gw).cpu()
        want = torch.zeros(8, E, dtype=torch.bool)
        for r in range(8):
            named = idx[r][idx[r] >= 0].cpu()
            bad = torch.isnan(x[r]).cpu()
            if score == "softmax" and not renorm:
                want[r] = len(named) > 0 and bool(bad.any())
            elif renorm:
                want[r, named] = bool(bad[named].any())
            else:
                want[r, named] = bad[named]
        assert torch.equal(torch.isnan(dx), want), (dtype, torch.isnan(dx).sum(1), want.sum(1))
        assert (dx[5] == 0).all()


@pytest.mark.parametrize("E", [64, 61, 250, 1024, 1030])
def test_route_backward_dense_of_distant_logits(E):
    """Softmax over all experts in fp32, scores far below the row's largest: the exponential's argument is
    off by 3 u for each unit of the distance (the difference, the factor log2 e, their product), the
    exponential, the sum and the products by some roundings; scores below the normal range are 0."""
    g = generator(E)
    K = 4
    x = torch.randn(64, E, generator=g, device=DEV) * 20
    rc = ep.RouteConfig(E=E, K=K, renormalize=False)
    idx, _ = ep.route(rc, x)
    gw = torch.rand(64, K, generator=g, device=DEV) + 0.5
    got = f64(ep.route_backward(rc, x, idx, gw))
    ref = plain.route_backward(rc, f64(x), idx.cpu().numpy(), f64(gw))
    rest = np.ones((64, E), bool)
    np.put_along_axis(rest, idx.cpu().numpy(), False, 1)
    # unchosen: -p sum(g p); the sum is off by what its largest scores are, whose distances are small or
    # whose part is (d exp(-d) < 0.37 for each of them)
    far = f64(x).max(1, keepdims=True) - f64(x)
    tol = np.abs(ref) * (3 * far + E / 8 + 40) * U + 2.0 ** -126 * 2
    over = np.where(rest, np.abs(got - ref) - tol, -1)
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


# -------------------------------------------------------------------------------- products

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,width", [(5, 64), (40, 64), (300, 4096 + 9), (600, 16385)])  # split, 128 and 256 rows a tile
def test_gates_that_close_and_open(dtype, M, width):
    """silu of gates down to where exp(gate) leaves fp32, times large ups: relative to the value as
    elsewhere.  The product's values are exact here (codes of one, scales of powers of two and gates
    themselves).  What silu itself has below the normal range is lost by half a step of fp32's smallest
    values, and for 16-bit results by scores below 2^-142, which count as 0."""
    t = DTYPES[dtype]
    K = 16
    gates = torch.cat([torch.linspace(-150, -75, M - M // 2, device=DEV), torch.linspace(-75, 200, M // 2, device=DEV)])
    a = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    a[:, 0] = 1
    w = torch.zeros(2 * width, K, dtype=torch.int8, device=DEV)
    w[:, 0] = 1
    ups = 2.0 ** (torch.arange(width, device=DEV) % 5 * 25 - 10.0)  # 2^-10 .. 2^90
    sw = torch.cat([torch.ones(width, device=DEV), ups])
    got = ep.matmul_int8((a, gates.contiguous()), (w, sw), gated=True, out_dtype=t).double()
    g = gates.double()[:, None]
    up = g * ups.double()[None, :]
    ref = g / (1 + torch.exp(-g)) * up
    rel = (4 * (1 + g.abs()) + 16) * U
    lost = 2.0 ** -149 if t == torch.float32 else 2.0 ** -142 * g.abs()
    # subnormal results: the last products lie on multiples of 2^-149, and bf16's subnormals are the multiples
    # of 2^-126 / 2^7 = 2^-133, fp16's of 2^-14 / 2^10 = 2^-24: a rounding to them is off by half of that
    step = {torch.float32: 2.0 ** -148, torch.bfloat16: 2.0 ** -134 + 2.0 ** -148, torch.float16: 2.0 ** -25}[t]
    tol = ref.abs() * (rel + half_step(t) * (1 + rel)) + lost * up.abs() + step
    if t == torch.float16:                            # beyond its largest value
        big = ref.abs() * (1 + rel) >= 65504
        assert (got.abs() >= 65504 * (1 - 2 * half_step(t)))[big].all()
        got, ref = torch.where(big, 0.0, got), torch.where(big, 0.0, ref)
    over = (got - ref).abs() - tol
    at = int(over.argmax())
    assert over.max() <= 0, (float(gates[at // width]), float(ups[at % width]), float(got.flatten()[at]), float(ref.flatten()[at]))
