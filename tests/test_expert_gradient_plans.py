"""Every way the gradients are cut: tiles of 256 and 128 rows, dense and by expert, over many steps, full and
half tiles in one stream, and slices of both gradients.  The plan is asserted, so that a case stays on its way.

Plain implementations and tolerances are those of test_expert_gradients.py."""

import numpy as np
import pytest
import torch

import combine_topk_idx_expert_amd as ep
from test_expert_gradients import case, close_product, np_or_none, product_gradient
from test_expert_products import (DEV, DROPPED, as_rows, assert_close, expected, f64, fp8_case, fp8_values, fp8_weights, gen,
                                  groups_of, half_case, spans)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def say(*a):
    print("[plans]", *a, flush=True)


# counts, inner, outer, (rows of a tile, slices) of the rows' gradient and of the weights'
GROUPED = {
    # tails of 1 to 128 and of 129 to 255 rows, full tiles between them, one row, none
    "tall": ([0, 1, 300, 129, 255, 700, 1000, 64, 513, 0, 380, 900, 2, 640, 257, 130], 1504, 1040, (256, 1), (256, 1)),
    "tall, few channels": ([0, 1, 300, 129, 255, 700, 1000, 64, 513, 0, 380, 900, 2, 640, 257, 130], 1504, 48, (256, 1), (128, 1)),
    "weights in slices": ([9000, 0, 1, 4000, 2500, 1500, 900, 112], 960, 288, (256, 1), (128, 2)),
    # slices that are empty for short groups, and end inside the long one's
    "weights in many slices": ([6000, 1, 0, 127, 64], 128, 128, (128, 1), (128, 9)),
    "weights in slices, odd": ([1, 3000, 0, 70, 6000, 129], 264, 144, (128, 1), (128, 7)),
    "rows in slices": ([100, 0, 30], 256, 4096, (128, 27), (128, 1)),
}


@pytest.mark.parametrize("name", list(GROUPED))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype,w32", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float16, True)])
def test_grouped_gradients_by_every_plan(name, gated, dtype, w32):
    counts, K, N, rows_plan, weights_plan = GROUPED[name]
    start, count, M = groups_of(counts, gap=3)
    G = len(counts)
    plan = ep.debug_backward_plan(M, G, K, N, gated)
    say(name, M, G, K, N, gated, dtype, w32, plan)
    assert plan == (rows_plan, weights_plan)
    a, w, grad, pre = case(G, M, K, N, G, gated, dtype)
    between = torch.ones(M, dtype=torch.bool, device=DEV)
    for s, n in spans(start, count):
        between[s:s + n] = False
    for t in (a, grad, pre):
        if t is not None:
            t[between] = float("nan")
    ga, gw = torch.full_like(a, 7.0), torch.full(w.shape, 7.0, dtype=torch.float32 if w32 else dtype, device=DEV)
    ep.matmul_backward(a, w, grad, rows=as_rows(start, count), gated=gated, pre=pre, out=(ga, gw))
    assert (ga[between] == 7.0).all()
    for e, (s, n) in enumerate(spans(start, count)):
        if n == 0:
            assert not gw[e].any()
            continue
        d, off = product_gradient(f64(grad[s:s + n]), None if pre is None else f64(pre[s:s + n]), dtype)
        close_product(ga[s:s + n], d, f64(w[e]).T.copy(), off, dtype, ("grad_a", e))
        close_product(gw[e], d.T.copy(), f64(a[s:s + n]).T.copy(), off.T.copy(), dtype, ("grad_w", e))


@pytest.mark.parametrize("M,K,N,plan", [(9000, 1504, 1040, ((256, 1), (128, 4))), (300, 3584, 4096, ((128, 5), (256, 1)))])
def test_dense_gradients_by_tall_tiles(M, K, N, plan):
    say("dense", M, K, N, ep.debug_backward_plan(M, 0, K, N))
    assert ep.debug_backward_plan(M, 0, K, N) == plan
    a, w, grad, pre = case(M, M, K, N, 0, False, torch.bfloat16)
    ga, gw = ep.matmul_backward(a, w, grad)
    d, off = product_gradient(f64(grad), np_or_none(pre), torch.bfloat16)
    close_product(ga, d, f64(w).T.copy(), off, torch.bfloat16, "grad_a")
    close_product(gw, d.T.copy(), f64(a).T.copy(), off.T.copy(), torch.bfloat16, "grad_w")


@pytest.mark.parametrize("K,N,gated", [(4096, 16, False), (16, 4096, True)])
@pytest.mark.parametrize("G", [0, 2])
def test_gradients_beyond_32_bits_of_offset(K, N, gated, G):
    """Rows, projections and slices past 2^32 bytes and elements; all rows but the first 200 and the last 300 are zeros."""
    M, n = (1 << 32) // 4096 + 300, 300
    dtype = torch.bfloat16
    plan = ep.debug_backward_plan(M, G, K, N, gated)
    say("far", M, K, N, gated, G, plan)
    assert plan[1][1] > 1
    far = lambda width: torch.zeros(M, width, dtype=dtype, device=DEV)
    a, grad, pre = far(K), far(N // 2 if gated else N), far(N) if gated else None
    ends = [slice(0, 200), slice(M - n, M)]
    for k, t in enumerate((a, grad, pre)):
        if t is not None:
            for s in ends:
                t[s] = torch.randn(t[s].shape, generator=gen(k + 1 + (s.start or 0)), device=DEV)
    w = (torch.randn((max(G, 1), N, K), generator=gen(9), device=DEV) / K ** 0.5).to(dtype)
    rows = as_rows([0, M - n], [200, n]) if G else None
    ga, gw = torch.full((M, K), 7.0, dtype=dtype, device=DEV), torch.empty((max(G, 1), N, K), dtype=torch.float32, device=DEV)
    ep.matmul_backward(a, w if G else w[0], grad, rows=rows, gated=gated, pre=pre, out=(ga, gw if G else gw[0]))
    at = lambda t, s: None if t is None else f64(t[s])
    parts = [product_gradient(at(grad, s), at(pre, s), dtype) for s in ends]
    for k, s in enumerate(ends):
        d, off = parts[k]
        close_product(ga[s], d, f64(w[k if G else 0]).T.copy(), off, dtype, ("grad_a", k))
        if G:
            close_product(gw[k], d.T.copy(), f64(a[s]).T.copy(), off.T.copy(), dtype, ("grad_w", k))
    middle = ga[200:M - n]
    assert (middle == 7.0).all() if G else not middle.any()
    if not G:
        d, off = (np.concatenate([p[i] for p in parts]).T.copy() for i in (0, 1))
        x = np.concatenate([f64(a[s]) for s in ends]).T.copy()
        close_product(gw[0], d, x, off, dtype, "grad_w")


def test_a_product_by_every_kernel():
    """Dense heights by rounds, and groups of few and of many rows side by side."""
    for M, K, N, gated, kernels in ((22240, 128, 326, True, ("tiles256",)), (65, 256, 49152, False, ("tiles128",)),
                                    (2300, 640, 6150, False, ("tiles256",)), (1003, 1024, 7168, False, ("tiles128",))):
        say("product", M, K, N, gated, kernels)
        assert ep.debug_product_kernels(M, 0, N, gated) == kernels
        a, sa, w, sw = fp8_case(1, M, K, N, 0, gated, False)
        x, v = fp8_values(a, sa, False), fp8_weights(w, sw, gated)
        ref, tol, _, _ = expected(x, v, gated, torch.bfloat16, DROPPED)
        assert_close(ep.matmul_fp8((a, sa), (w, sw), gated=gated), ref, tol, "fp8")
        a, w = half_case(2, M, K, N, 0, torch.float16)
        ref, tol, _, _ = expected(f64(a), f64(w), gated, torch.float16)
        assert_close(ep.matmul(a, w, gated=gated), ref, tol, "half")
