"""Gradients of the 16-bit product against plain 64-bit implementations.

Tolerances as in test_expert_products.py; gated, the product's gradient d is rounded to the rows' type
before it enters the other two: half a step of |d|, and some roundings of its own terms.
"""

import numpy as np
import pytest
import torch

import combine_topk_idx_expert_amd as ep
import plain_expert_layer as plain
from test_expert_products import DEV, TINY, U, as_rows, assert_close, f64, gen, groups_of, half_case, spans, times

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def say(*a):
    print("[gradients]", *a, flush=True)


def product_gradient(grad, pre, dtype):
    """(d, bound of its error), float64."""
    if pre is None:
        return grad, np.zeros_like(grad)
    d = plain.gate_backward(pre, grad)
    half = pre.shape[1] // 2
    g, u = np.abs(pre[:, :half]), np.abs(pre[:, half:])
    # the sigmoid is off by some 2^-22 (its exponent's argument by |g| u), and 1 - s as much absolutely
    s_off = 2.0 ** -21 + np.minimum(g, 110) * 2 * U
    own = np.concatenate([np.abs(grad) * u * (1 + g), np.abs(grad) * g], 1) * np.concatenate([s_off * (1 + g), s_off], 1)
    return d, own + (torch.finfo(dtype).eps / 2) * np.abs(d) + TINY[dtype]


def close_product(got, x, y, x_off, dtype, what):
    """got = x @ y.T, x off by x_off."""
    ref, size = times(x, y, None)
    _, off = times(x_off, y, None)
    tol = (2 * x.shape[1] + 16) * U * (size + off) + off + (torch.finfo(got.dtype).eps / 2 + U) * np.abs(ref) + TINY[got.dtype]
    assert_close(got, ref, tol, what)


def case(seed, M, K, N, G, gated, dtype):
    a, w = half_case(seed, M, K, N, G, dtype)
    g = gen(seed + 1)
    grad = torch.randn((M, N // 2 if gated else N), generator=g, device=DEV).to(dtype)
    pre = (2 * torch.randn((M, N), generator=g, device=DEV)).to(dtype) if gated else None
    return a, w, grad, pre


def np_or_none(t):
    return None if t is None else f64(t)


SHAPES = [(1, 8, 16), (1, 512, 64), (3, 24, 48), (31, 264, 272), (32, 128, 128), (33, 72, 80), (64, 520, 640), (130, 1032, 304),
          (257, 256, 256), (300, 2056, 528), (1003, 512, 1040), (2100, 784, 2064), (4096, 2048, 512)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_dense_gradients_match_plain(M, K, N, gated):
    for dtype, w32 in ((torch.bfloat16, False), (torch.float16, True)):
        say(M, K, N, gated, dtype, w32)
        a, w, grad, pre = case(M, M, K, N, 0, gated, dtype)
        out = (torch.empty_like(a), torch.empty(N, K, dtype=torch.float32, device=DEV)) if w32 else None
        ga, gw = ep.matmul_backward(a, w, grad, gated=gated, pre=pre, out=out)
        assert ga.dtype == dtype and gw.dtype == (torch.float32 if w32 else dtype)
        d, off = product_gradient(f64(grad), np_or_none(pre), dtype)
        close_product(ga, d, f64(w).T.copy(), off, dtype, "grad_a")
        close_product(gw, d.T.copy(), f64(a).T.copy(), off.T.copy(), dtype, "grad_w")


GROUPS = [
    ([3, 0, 2, 1], 256, 96),
    ([0, 0, 0], 64, 32),
    ([1], 72, 144),
    ([17, 64, 65, 0, 130, 5], 520, 528),
    ([128, 129, 255, 256, 257, 300], 136, 1312),
    ([700, 1, 0, 520, 64, 900, 33], 2312, 320),
    (list(range(0, 70)), 40, 48),
    ([2000, 3000, 0, 1500, 20], 264, 2064),
]


@pytest.mark.parametrize("counts,K,N", GROUPS, ids=[str(i) for i in range(len(GROUPS))])
@pytest.mark.parametrize("gated", [False, True])
def test_group_gradients_match_plain(counts, K, N, gated):
    start, count, M = groups_of(counts, gap=3)
    G = len(counts)
    for dtype in (torch.bfloat16, torch.float16):
        say("groups", G, K, N, gated, dtype)
        a, w, grad, pre = case(G, M, K, N, G, gated, dtype)
        # what lies between the groups is NaN: it may not reach any row or weight
        between = torch.ones(M, dtype=torch.bool, device=DEV)
        for s, n in spans(start, count):
            between[s:s + n] = False
        for t in (a, grad, pre):
            if t is not None:
                t[between] = float("nan")
        ga, gw = torch.full_like(a, 7.0), torch.full_like(w, 7.0)
        ep.matmul_backward(a, w, grad, rows=as_rows(start, count), gated=gated, pre=pre, out=(ga, gw))
        assert (ga[between] == 7.0).all()
        for e, (s, n) in enumerate(spans(start, count)):
            if n == 0:
                assert not gw[e].any()
                continue
            d, off = product_gradient(f64(grad[s:s + n]), None if pre is None else f64(pre[s:s + n]), dtype)
            close_product(ga[s:s + n], d, f64(w[e]).T.copy(), off, dtype, ("grad_a", e))
            close_product(gw[e], d.T.copy(), f64(a[s:s + n]).T.copy(), off.T.copy(), dtype, ("grad_w", e))


@pytest.mark.parametrize("M,K,N", [(30000, 1000, 64), (20000, 1024, 128), (9000, 1504, 192)])
def test_rows_of_few_channels_over_many_tiles(M, K, N):
    """One, two and three steps a tile of the rows' gradient, more tiles than workgroups."""
    a, w, grad, _ = case(1, M, K, N, 0, False, torch.bfloat16)
    ga, gw = ep.matmul_backward(a, w, grad, out=(torch.empty_like(a), torch.empty(N, K, device=DEV)))
    d, off = product_gradient(f64(grad), None, torch.bfloat16)
    close_product(ga, d, f64(w).T.copy(), off, torch.bfloat16, "grad_a")
    close_product(gw, d.T.copy(), f64(a).T.copy(), off.T.copy(), torch.bfloat16, "grad_w")


@pytest.mark.parametrize("counts,K,N", [([40, 64, 65, 128, 1, 0, 130, 200] * 4, 1024, 1024), ([1, 0, 2] * 1365, 24, 32)],
                         ids=["many tiles", "many groups"])
def test_weights_of_groups_of_few_rows(counts, K, N):
    start, count, M = groups_of(counts)
    G = len(counts)
    a, w, grad, pre = case(2, M, K, N, G, True, torch.bfloat16)
    ga, gw = ep.matmul_backward(a, w, grad, rows=as_rows(start, count), gated=True, pre=pre)
    for e, (s, n) in enumerate(spans(start, count)):
        if n == 0:
            assert not gw[e].any()
            continue
        d, off = product_gradient(f64(grad[s:s + n]), f64(pre[s:s + n]), torch.bfloat16)
        close_product(ga[s:s + n], d, f64(w[e]).T.copy(), off, torch.bfloat16, ("grad_a", e))
        close_product(gw[e], d.T.copy(), f64(a[s:s + n]).T.copy(), off.T.copy(), torch.bfloat16, ("grad_w", e))


@pytest.mark.parametrize("gated", [False, True])
def test_one_gradient_without_the_other_and_no_rows(gated):
    for rows in (None, as_rows([0, 100], [90, 0])):
        G = 0 if rows is None else 2
        a, w, grad, pre = case(5, 100, 136, 64, G, gated, torch.bfloat16)
        ga, gw = torch.zeros_like(a), torch.zeros_like(w)
        ep.matmul_backward(a, w, grad, rows=rows, gated=gated, pre=pre, out=(ga, gw))
        for one in ((torch.zeros_like(a), None), (None, torch.zeros_like(w))):
            got = ep.matmul_backward(a, w, grad, rows=rows, gated=gated, pre=pre, out=one)
            for x, y in zip(got, (ga, gw)):
                assert x is None or torch.equal(x, y)
        none = [t[:0] if t is not None else None for t in (a, grad, pre)]
        gx, gw = ep.matmul_backward(none[0], w, none[1], rows=rows, gated=gated, pre=none[2],
                                    out=(none[0].clone(), torch.full_like(w, 7.0)))
        assert gx.shape[0] == 0 and not gw.any()


def test_gates_at_the_ends():
    """Gates whose exponential leaves fp32, and zeros."""
    dtype = torch.bfloat16
    v = [0.0, -0.0, 1e-3, -1.28, 20.0, -20.0, 88.0, -88.0, 120.0, -120.0, 3e4, -3e4, 1e30, -1e30, 5.0, -5.0]
    g = torch.tensor(v, device=DEV).repeat(16, 1).to(dtype)
    u = torch.randn(16, 16, generator=gen(1), device=DEV).to(dtype)
    pre = torch.cat([g, u], 1).contiguous()
    grad = torch.randn(16, 16, generator=gen(2), device=DEV).to(dtype)
    a = torch.eye(16, device=DEV).to(dtype)
    w = torch.zeros(32, 16, device=DEV, dtype=dtype)
    _, gw = ep.matmul_backward(a, w, grad, gated=True, pre=pre, out=(None, torch.empty(32, 16, device=DEV)))
    d, off = product_gradient(f64(grad), f64(pre), dtype)
    assert_close(gw.t(), d, off, "d")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gates_that_were_rounded_to_infinities(dtype):
    """Their gate is shut or open; NaN stays NaN."""
    pre = torch.zeros(8, 16, device=DEV, dtype=dtype)
    pre[:, 8:] = 3.0
    pre[0, :8], pre[1, :8], pre[2, :8] = float("-inf"), float("inf"), float("nan")
    grad = torch.full((8, 8), 2.0, device=DEV, dtype=dtype)
    one = torch.zeros(1, 8, device=DEV, dtype=dtype)
    one[0, 0] = 1.0
    w = torch.zeros(16, 8, device=DEV, dtype=dtype)
    # a row at a time, since an infinity times another row's zero is NaN: column 0 of grad_w is its gradient
    for r, (dg, du) in enumerate([(0.0, 0.0), (6.0, float("inf")), (float("nan"), float("nan")), (3.0, 0.0)]):
        _, g = ep.matmul_backward(one, w, grad[r:r + 1], gated=True, pre=pre[r:r + 1].contiguous(),
                                  out=(None, torch.empty(16, 8, device=DEV)))
        np.testing.assert_allclose(f64(g[:8, 0]), np.full(8, dg))
        np.testing.assert_allclose(f64(g[8:, 0]), np.full(8, du))


def test_gradients_agree_with_differences():
    """Forward and backward pass along random directions of the 64-bit function."""
    r = np.random.default_rng(1)
    M, K, N, dtype = 40, 64, 48, torch.bfloat16
    a, w = half_case(3, M, K, N, 0, dtype)
    c = torch.randn(M, N // 2, generator=gen(4), device=DEV).to(dtype)
    pre = torch.empty(M, N, dtype=dtype, device=DEV)
    ep.matmul(a, w, gated=True, pre=pre)
    ga, gw = ep.matmul_backward(a, w, c, gated=True, pre=pre)
    x, v, cc = f64(a), f64(w), f64(c)
    f = lambda x, v: (plain.gate(x @ v.T) * cc).sum()
    for _ in range(4):
        e, h, step = r.standard_normal(x.shape), r.standard_normal(v.shape), 1e-5
        slope = (f(x + step * e, v + step * h) - f(x - step * e, v - step * h)) / (2 * step)
        got = (f64(ga) * e).sum() + (f64(gw) * h).sum()
        # pre, d and the results are rounded to bf16, 2^-8 each at most: as independent errors of the terms
        # of both sums, with six deviations
        size = np.sqrt(((f64(ga) * e) ** 2).sum() + ((f64(gw) * h) ** 2).sum())
        assert abs(got - slope) < 6 * 3 * 2.0 ** -8 * size * 3


def test_gradients_on_streams_and_in_graphs():
    start, count, M = groups_of([130, 0, 70, 300])
    rows = as_rows(start, count)
    a, w, grad, _ = case(1, M, 256, 512, 4, True, torch.bfloat16)

    def step():
        pre, out = torch.zeros(M, 512, dtype=a.dtype, device=DEV), torch.zeros_like(grad)
        ep.matmul(a, w, rows=rows, gated=True, pre=pre, out=out)
        ga, gw = torch.zeros_like(a), torch.zeros_like(w)
        ep.matmul_backward(a, w, grad, rows=rows, gated=True, pre=pre, out=(ga, gw))
        return [out, pre, ga, gw]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        a.copy_(torch.randn(a.shape, generator=gen(60 + k), device=DEV))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_two_graphs_replayed_at_once():
    """Workspaces (the gate's gradient, slices, the norm's partial sums) belong to a graph each."""
    graphs = []
    for k in range(2):
        a, w, grad, pre = case(10 + k, 6000, 256, 512, 0, True, torch.bfloat16)
        wn = torch.ones(256, device=DEV)

        def step(a=a, w=w, grad=grad, pre=pre, wn=wn):
            ga, gw = ep.matmul_backward(a, w, grad, gated=True, pre=pre)
            return [ga, gw, *ep.rms_norm_backward(a, wn, ga)]

        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, want, torch.cuda.Stream(), step))  # (step holds the inputs that the graph reads)
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, out, _, stream, _ in graphs:
            with torch.cuda.stream(stream):
                for t in out:
                    t.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _ in graphs:
            assert all(torch.equal(x, y) for x, y in zip(out, want))
