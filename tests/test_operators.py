"""Routing, int8 quantising and the int8 products against plain 64-bit implementations.

Tolerances come from the number of roundings; u is half a step of fp32, 2^-24.  Ids, codes and
row scales are whole numbers or single correctly rounded quotients and are compared for
equality.
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


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def say(*a):
    print("[operators]", *a, flush=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def assert_close(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    over = np.abs(np.nan_to_num(got) - np.nan_to_num(ref)) - tol
    assert over.max(initial=-1.0) <= 0, (what, over.max(), np.unravel_index(over.argmax(), over.shape))


# -------------------------------------------------------------------------------- routing

ROUTERS = [
    # E, K, groups, kept groups, group score
    (256, 8, 1, 1, "max"),
    (256, 8, 8, 4, "top2"),
    (256, 6, 8, 3, "max"),
    (256, 8, 4, 2, "top2"),
    (128, 8, 1, 1, "max"),
    (128, 4, 16, 5, "top2"),
    (512, 8, 8, 4, "top2"),
    (160, 6, 8, 3, "top2"),
    (64, 6, 1, 1, "max"),
    (60, 4, 1, 1, "max"),
    (61, 5, 1, 1, "max"),
    (16, 2, 4, 2, "max"),
    (16, 16, 1, 1, "max"),
    (8, 1, 8, 3, "top2"),
    (1, 1, 1, 1, "max"),
    (384, 8, 1, 1, "max"),
    (320, 10, 64, 7, "top2"),
    (1000, 32, 1, 1, "max"),
    (4096, 32, 64, 9, "top2"),
    # more than eight choices, and groups that do not share their experts evenly among lanes
    (256, 10, 1, 1, "max"),
    (256, 16, 8, 4, "top2"),
    (61, 9, 1, 1, "max"),
    (16, 10, 1, 1, "max"),
    (512, 12, 8, 4, "top2"),
    (492, 2, 4, 4, "max"),
    (488, 10, 8, 5, "top2"),
    (216, 5, 8, 6, "top2"),
    (204, 8, 4, 3, "max"),
    (312, 9, 8, 4, "top2"),
    (255, 8, 3, 2, "top2"),
    (54, 11, 6, 3, "top2"),
    (12, 3, 4, 3, "top2"),
    (72, 8, 8, 8, "max"),
    (239, 8, 1, 1, "max"),
    (137, 6, 1, 1, "max"),
    (9, 9, 1, 1, "max"),
    (128, 8, 4, 4, "top2"),
]


def router(E, K, groups=1, kept=1, group_score="max", score="softmax", renormalize=True, scale=1.0):
    return ep.RouteConfig(E=E, K=K, score=score, num_groups=groups, topk_groups=kept, group_score=group_score,
                          renormalize=renormalize, scale=scale)


def weight_tolerance(x, K, scale):
    """Relative: the argument of exp is off by a few u for each unit of its size (the difference to the
    largest logit, the factor log2 e), the exponential, the quotient and the sum over up to E scores in a
    tree add some roundings more."""
    top = np.abs(np.where(np.isfinite(x), x, 0)).max()
    return (40 + K + 8 * min(top, 110)) * U * scale


def check_route(rc, logits, bias=None, mask=None):
    x = f64(logits)
    idx, w = ep.route(rc, logits, bias=bias, token_mask=mask)
    ref_idx, ref_w = plain.route(rc, x, None if bias is None else f64(bias), None if mask is None else mask.cpu().numpy())
    np.testing.assert_array_equal(idx.cpu().numpy(), ref_idx)
    tol = weight_tolerance(x, rc.K, 1.0)
    assert_close(f64(w), ref_w, tol * np.nan_to_num(np.abs(ref_w)) + 2.0 ** -125, "weights")
    return idx, w


@pytest.mark.parametrize("E,K,groups,kept,group_score", ROUTERS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_matches_plain(E, K, groups, kept, group_score, score):
    g = torch.Generator(device=DEV).manual_seed(E * 100 + K)
    for n, (T, dtype, with_bias, renorm, with_mask) in enumerate([
            (1, "fp32", True, True, False), (37, "bf16", False, True, True), (129, "fp16", True, False, False),
            (200, "bf16", True, True, True), (65, "fp32", False, False, False)]):
        say("route", E, K, groups, kept, group_score, score, T, dtype, with_bias, renorm, with_mask)
        rc = router(E, K, groups, kept, group_score, score, renorm, 2.5 if n % 2 else 1.0)
        x = (torch.randn(T, E, generator=g, device=DEV) * 1.5).to(DTYPES[dtype])
        width = 0.05 if score == "sigmoid" else 0.2 / E
        bias = torch.randn(E, generator=g, device=DEV) * width if with_bias else None
        mask = torch.rand(T, generator=g, device=DEV) < 0.8 if with_mask else None
        check_route(rc, x, bias, mask)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,group_score", [(1, 1, "max"), (8, 4, "top2"), (8, 3, "max")])
@pytest.mark.parametrize("E,K", [(256, 8), (256, 13), (216, 8), (200, 16)])
def test_route_ties_go_to_the_lowest_expert(score, groups, kept, group_score, E, K):
    """Logits of few values, a zero bias, signed zeros, equal rows: ties everywhere."""
    g = torch.Generator(device=DEV).manual_seed(3)
    rc = router(E, K, groups, kept, group_score, score)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randint(-2, 3, (300, E), generator=g, device=DEV).to(dtype)
        x[0] = 0.0
        x[1, ::2] = -0.0
        x[2] = 7.0
        for bias in (None, torch.zeros(E, device=DEV), torch.randint(0, 2, (E,), generator=g, device=DEV) * 0.125,
                     torch.randint(-3, 1, (E,), generator=g, device=DEV) * 0.5):  # keys below zero
            check_route(rc, x, bias)


def test_route_orders_scores_that_fp32_merges():
    """Keys that differ by less than a step of fp32 keep the order of exact arithmetic: one expert's
    score is that of another plus a difference of 2^-26 in its logit's score, under a bias that hides it."""
    g = torch.Generator(device=DEV).manual_seed(4)
    T, E = 512, 256
    x = torch.randn(T, E, generator=g, device=DEV) * 0.3 + 2.0
    # bias moves every expert to about the same key: the keys of a row lie within a few fp32 steps
    base = torch.linspace(1.0, 3.0, E, device=DEV)
    x = base.repeat(T, 1)
    step = torch.randint(-3, 4, (T, E), generator=g, device=DEV)
    x = (x.view(torch.int32) + step.int()).view(torch.float32)
    bias = (0.5 - torch.sigmoid(base.double())).float()
    for groups, kept, gscore in ((1, 1, "max"), (8, 4, "top2"), (8, 4, "max")):
        for K in (8, 12):
            check_route(router(E, K, groups, kept, gscore, "sigmoid"), x, bias)
    p = torch.softmax(base.double(), 0)
    check_route(router(E, 8, 1, 1, "max", "softmax"), x, (0.01 - p).float())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,K", [(256, 1, 1, 8), (256, 8, 2, 8), (61, 1, 1, 8), (1000, 8, 2, 8),
                                             (256, 8, 2, 11), (61, 1, 1, 16), (204, 4, 2, 8), (312, 8, 3, 10)])
def test_route_masked_infinite_and_nan_logits(score, E, groups, kept, K):
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(24, E, generator=g, device=DEV)
    inf = float("inf")
    x[0] = -inf                       # nothing to choose
    x[1] = -inf
    x[1, E // 2] = 1.0                # one to choose
    x[2, : E - 3] = -inf              # three to choose
    x[3, 5] = inf                     # the largest
    x[4, 5] = x[4, 3] = inf           # tied
    x[5, 7] = float("nan")
    x[6] = float("nan")
    x[7] = -inf
    x[7, 2] = float("nan")
    x[8] = -3.0e38
    x[9] = 3.4e38
    x[10] = -120.0 - torch.arange(E, device=DEV) * 0.01  # scores that underflow
    x[11] = torch.where(torch.rand(E, generator=g, device=DEV) < 0.5, -inf, x[11])
    x[12, ::2] = float("nan")
    x[13, 0] = -inf
    bias = torch.randn(E, generator=g, device=DEV) * 0.01
    wild = bias.clone()
    wild[1], wild[4], wild[9] = -inf, inf, float("nan")
    for renorm in (True, False):
        rc = router(E, K, groups, kept, "top2" if groups > 1 else "max", score, renorm)
        for b in (None, bias, wild):
            say("wild", E, groups, score, renorm, b is None)
            check_route(rc, x, b)
            check_route(rc, x[:14].to(torch.bfloat16), b)


def test_route_rows_apart_unaligned_and_given_outputs():
    g = torch.Generator(device=DEV).manual_seed(6)
    for E, dtype in ((256, torch.float32), (256, torch.bfloat16), (64, torch.float16), (61, torch.bfloat16)):
        wide = torch.randn(70, E + 13, generator=g, device=DEV).to(dtype)
        for off in (0, 1, 8):
            x = wide[:, off:off + E]
            rc = router(E, 5, score="sigmoid")
            out = (torch.full((70, 5), -7, dtype=torch.int64, device=DEV), torch.full((70, 5), 9.0, device=DEV))
            idx, w = ep.route(rc, x, out=out)
            assert idx is out[0] and w is out[1]
            again = ep.route(rc, x.contiguous())
            assert torch.equal(idx, again[0]) and torch.equal(w, again[1])
            gw = torch.randn(70, 5, generator=g, device=DEV)
            assert torch.equal(ep.route_backward(rc, x, idx, gw), ep.route_backward(rc, x.contiguous(), idx, gw))
    empty = ep.route(router(16, 2), torch.empty(0, 16, device=DEV))
    assert empty[0].shape == (0, 2) and empty[1].shape == (0, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,K", [(256, 8), (256, 6), (61, 5), (16, 16), (8, 1), (512, 10), (1000, 32), (4096, 32)])
def test_route_backward_matches_the_formula(score, renorm, E, K):
    g = torch.Generator(device=DEV).manual_seed(E + K)
    for T, dtype in ((1, torch.float32), (133, torch.bfloat16), (70, torch.float32), (67, torch.float16)):
        say("route_backward", score, renorm, E, K, T, dtype)
        x = (torch.randn(T, E, generator=g, device=DEV) * 1.5).to(dtype)
        rc = router(E, K, score=score, renormalize=renorm, scale=2.5)
        idx, w = ep.route(rc, x)
        if T > 4:
            idx[1] = -1                      # an unrouted token
            idx[2, K - 1] = -1               # an unused slot
            idx[3, 0] = idx[3, K - 1]        # an expert named twice
            idx[4, 0] = E + 5                # outside: unused
        gw = torch.randn(T, K, generator=g, device=DEV)
        dx = ep.route_backward(rc, x, idx, gw)
        assert dx.dtype == dtype and dx.shape == x.shape
        ref = plain.route_backward(rc, f64(x), idx.cpu().numpy(), f64(gw))
        # every term is a weight (at most `scale`, with the tolerance of the weights) times sums of K
        # gradients, each rounding of which counts against the largest of them
        big = np.abs(f64(gw)).max(1, keepdims=True)
        tol = (weight_tolerance(f64(x), K, 1.0) + 4 * K * U) * 2.5 * 2 * big + half_step(dtype) * np.abs(ref)
        if dtype == torch.float16:
            tol = tol + 2.0 ** -25           # half a step of its subnormals
        assert_close(f64(dx), ref, tol, "grad")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False)])
@pytest.mark.parametrize("E,K", [(61, 4), (137, 12), (256, 8), (600, 6), (1030, 5)])
def test_route_backward_at_any_address(dtype, score, renorm, E, K):
    """Logits and gradients that start at any element, nothing written beside them."""
    g = torch.Generator(device=DEV).manual_seed(E + K)
    T = 43
    rc = router(E, K, score=score, renormalize=renorm)
    x = torch.randn(T, E, generator=g, device=DEV).to(DTYPES[dtype])
    idx, _ = ep.route(rc, x)
    gw = torch.randn(T, K, generator=g, device=DEV)
    want = ep.route_backward(rc, x, idx, gw)
    for off in (1, 3):
        rows = torch.empty(T * (E + 3) + off, dtype=DTYPES[dtype], device=DEV)[off:].view(T, E + 3)[:, :E]
        rows.copy_(x)
        store = torch.full((T * E + 32,), 9.0, dtype=DTYPES[dtype], device=DEV)
        grad = store[off:off + T * E].view(T, E)
        ep.route_backward(rc, rows, idx, gw, out=grad)
        assert torch.equal(grad, want)
        assert (store[:off] == 9.0).all() and (store[off + T * E:] == 9.0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_matches_differences(score, renorm):
    """Central differences of the 64-bit weights: h^2 times third derivatives (at most about 6 scale),
    and 2^-52 / h of rounding."""
    rng = np.random.default_rng(8)
    T, E, K, h = 6, 24, 4, 1e-4
    rc = router(E, K, score=score, renormalize=renorm, scale=1.5)
    x = rng.standard_normal((T, E)).astype(np.float32)
    idx, _ = plain.route(rc, x)
    gw = rng.standard_normal((T, K)).astype(np.float32)
    num = np.zeros((T, E))
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        up = plain.weights(rc, x.astype(np.float64) + d, idx)
        down = plain.weights(rc, x.astype(np.float64) - d, idx)
        num[:, e] = ((up - down) * gw).sum(1) / (2 * h)
    got = ep.route_backward(rc, torch.from_numpy(x).to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(gw).to(DEV))
    tol = 10 * 1.5 * K * h * h + 1e-11 + weight_tolerance(x, K, 1.0) * 1.5 * 8
    assert_close(f64(got), num, tol + np.zeros((T, E)), "grad against differences")


def test_route_backward_extreme_logits():
    inf = float("inf")
    x = torch.zeros(6, 16, device=DEV)
    x[0] = -inf
    x[1, 3] = -inf
    x[2] = -130.0 - torch.arange(16, device=DEV)
    x[3] = 100.0 + torch.arange(16, device=DEV)
    x[4, 5] = inf
    x[5, ::2] = -inf
    gw = torch.linspace(-1, 2, 24, device=DEV).view(6, 4)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            rc = router(16, 4, score=score, renormalize=renorm)
            idx, _ = ep.route(rc, x)
            got = f64(ep.route_backward(rc, x, idx, gw))
            ref = plain.route_backward(rc, f64(x), idx.cpu().numpy(), f64(gw))
            ref[0] = 0.0  # no choice, no gradient
            tol = (40 + 4 + 8 * 145) * U * 4
            assert np.isfinite(got).all()
            assert_close(got, ref, tol + np.zeros_like(ref), (score, renorm))


# ------------------------------------------------------------------------------ quantising

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 16), (2, 61), (130, 128), (17, 520), (9, 1000), (3, 2048),
                                       (70, 4096), (33, 7168), (4, 8192), (2, 12296), (2, 40000)])
def test_quantize_matches_plain(dtype, rows, cols):
    say("quantize", dtype, rows, cols)
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device=DEV) * torch.exp(torch.randn(rows, 1, generator=g, device=DEV))
    x = x.to(DTYPES[dtype])
    codes, scales = ep.quantize_int8(x)
    ref_codes, ref_scales = plain.quantize(f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), ref_scales)
    np.testing.assert_array_equal(codes.cpu().numpy(), ref_codes)
    wide = torch.zeros(rows, cols + 5, dtype=DTYPES[dtype], device=DEV)
    for off in (0, 3):  # rows apart, aligned to nothing
        wide[:, off:off + cols] = x
        again = ep.quantize_int8(wide[:, off:off + cols], out=(torch.full_like(codes, 99), torch.full_like(scales, 9.0)))
        assert torch.equal(again[0], codes) and torch.equal(again[1], scales)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 61), (5, 520), (1030, 2048), (2, 16392)])
def test_quantize_writes_its_rows_alone(dtype, rows, cols):
    """Codes that start at any byte, in the midst of others."""
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device=DEV).to(DTYPES[dtype])
    want = ep.quantize_int8(x)
    for off in (1, 7):
        store = torch.full((rows * cols + 32,), 99, dtype=torch.int8, device=DEV)
        codes = store[off:off + rows * cols].view(rows, cols)
        got = ep.quantize_int8(x, out=(codes, torch.empty(rows, device=DEV)))
        assert torch.equal(codes, want[0]) and torch.equal(got[1], want[1])
        assert (store[:off] == 99).all() and (store[off + rows * cols:] == 99).all()


def test_quantize_borders_and_odd_values():
    inf, nan = float("inf"), float("nan")
    for dtype in DTYPES.values():
        for cols in (512, 509):
            x = torch.zeros(14, cols, device=DEV)
            x[1] = -0.0
            x[2, 5] = nan
            x[3, 5] = inf
            x[4, 5] = -inf
            # scale 1: quotients on the border between two codes, ties to even
            x[5] = (torch.arange(cols, device=DEV) % 254 - 127) / 2.0
            x[5, 0] = 127.0
            # scale 2^-3
            x[6] = (torch.arange(cols, device=DEV) % 509 - 254) / 16.0
            x[6, 0] = -127 / 8
            x[7, 3] = torch.finfo(dtype).tiny
            x[8] = torch.finfo(dtype).tiny * torch.rand(cols, device=DEV)
            x[9] = torch.finfo(dtype).max
            x[10] = -torch.finfo(dtype).max * torch.rand(cols, device=DEV)
            x[11, cols - 1] = -1.0
            x[12, 0] = 1e-30
            x[13] = torch.randn(cols, device=DEV)
            x = x.to(dtype)
            x[7, 0] = torch.tensor(1, dtype=torch.int16 if dtype != torch.float32 else torch.int32).view(dtype)  # smallest subnormal
            codes, scales = ep.quantize_int8(x)
            ref_codes, ref_scales = plain.quantize(f64(x))
            np.testing.assert_array_equal(scales.cpu().numpy(), ref_scales)
            np.testing.assert_array_equal(codes.cpu().numpy(), ref_codes)


def test_quantize_near_borders_fp32():
    """fp32 values one step to either side of a border between two codes."""
    for top in (1.0, 127.0, 0.7310585, 3.3e-5):
        scale = np.float32(top) / np.float32(127)
        k = np.arange(-126, 127, dtype=np.float64)
        mid = ((k + 0.5) * np.float64(scale)).astype(np.float32)
        x = np.concatenate([mid, np.nextafter(mid, np.float32(9)), np.nextafter(mid, np.float32(-9)), [top]])
        x = np.tile(x.astype(np.float32), (3, 1))
        codes, scales = ep.quantize_int8(torch.from_numpy(x).to(DEV))
        ref_codes, ref_scales = plain.quantize(x)
        np.testing.assert_array_equal(scales.cpu().numpy(), ref_scales)
        np.testing.assert_array_equal(codes.cpu().numpy(), ref_codes)


# -------------------------------------------------------------------------------- products

def codes(g, *shape, extreme=False):
    if extreme:
        return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, -128, 127).to(torch.int8)
    return torch.randint(-128, 128, shape, generator=g, device=DEV).to(torch.int8)


def product_tolerance(ref, gate, dtype):
    """fp32 value of the sum, two scales: three roundings; a gate's silu is off by those times
    1 + |gate|, its exponential, quotient and the last product by a few more, and the result is rounded to the
    output's type.  Below the normal range of fp32 a rounding is up to 2^-150."""
    rel = 3.1 * U if gate is None else (4 * (1 + np.abs(gate)) + 16) * U
    tol = np.abs(ref) * (rel + half_step(dtype) * (1 + rel)) + 2.0 ** -148
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    return tol


def check_product(g, M, K, N, counts, starts, gated, dtype, extreme=False):
    G = 0 if counts is None else len(counts)
    a = codes(g, M, K, extreme=extreme)
    w = codes(g, *((G, N, K) if G else (N, K)), extreme=extreme)
    sa = (torch.rand(M, generator=g, device=DEV) + 0.5) * 2.0 ** -7
    sw = (torch.rand(w.shape[:-1], generator=g, device=DEV) + 0.5) * 2.0 ** -7 / K ** 0.5
    width = N // 2 if gated else N
    out = torch.full((M, width), -77.0, dtype=dtype, device=DEV)
    rows = None
    if G:
        rows = (torch.tensor(starts, dtype=torch.int64, device=DEV), torch.tensor(counts, dtype=torch.int32, device=DEV))
    got = ep.matmul_int8((a, sa), (w, sw), rows=rows, gated=gated, out=out)
    assert got is out
    got = f64(got)
    ref = np.full((M, width), -77.0)
    gate = np.zeros((M, width)) if gated else None
    an, wn, san, swn = a.cpu().numpy(), w.cpu().numpy(), sa.cpu().numpy(), sw.cpu().numpy()
    for e in range(max(G, 1)):
        lo, n = (starts[e], counts[e]) if G else (0, M)
        if n <= 0 or lo < 0 or lo >= M:
            continue
        hi = min(lo + n, M)
        y, gv = plain.product(an[lo:hi], san[lo:hi], wn[e] if G else wn, swn[e] if G else swn, gated)
        ref[lo:hi] = y
        if gated:
            gate[lo:hi] = gv
    assert_close(got, ref, product_tolerance(ref, gate, dtype), (M, K, N, counts, gated, dtype))


DENSE = [
    # rows, inner, outer
    (1, 16, 2), (1, 7168, 512), (2, 64, 6), (3, 2048, 130), (15, 144, 34), (16, 512, 64), (17, 1040, 256), (33, 256, 100),
    (64, 128, 128), (65, 400, 514), (130, 192, 258), (200, 1024, 1536), (257, 2064, 512), (300, 384, 770),
    (513, 640, 1026), (1003, 256, 514), (1025, 144, 300),
]


@pytest.mark.parametrize("M,K,N", DENSE)
@pytest.mark.parametrize("gated", [False, True])
def test_product_dense_matches_plain(M, K, N, gated):
    g = torch.Generator(device=DEV).manual_seed(M + K + N)
    for dtype in (torch.bfloat16, torch.float32) if M != 200 else DTYPES.values():
        say("product dense", M, K, N, gated, dtype)
        check_product(g, M, K, N, None, None, gated, dtype)
    if not gated:
        say("product dense", M, K, N + 1, "odd")
        check_product(g, M, K, N + 1, None, None, gated, torch.bfloat16)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,width", [
    (1, 2048, 4091), (5, 2064, 16384), (40, 2048, 4091), (64, 2048, 8190), (250, 2304, 4093),  # streams of weights
    (300, 208, 8188), (600, 208, 16385),                                                       # tiles
])
def test_product_wide_matches_plain(M, K, width, gated):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    N = width * (2 if gated else 1)
    a, w = codes(g, M, K), codes(g, N, K)
    sa = (torch.rand(M, generator=g, device=DEV) + 0.5) * 2.0 ** -7
    sw = (torch.rand(N, generator=g, device=DEV) + 0.5) * 2.0 ** -7 / K ** 0.5
    ref = f64(a.double() @ w.double().t().contiguous()) * f64(sa)[:, None] * f64(sw)[None, :]  # (sums below 2^53: exact)
    gate = None
    if gated:
        gate, up = ref[:, :width], ref[:, width:]
        ref = plain.silu(gate) * up
    for dtype in (torch.bfloat16, torch.float32):
        say("product wide", M, K, width, gated, dtype)
        got = ep.matmul_int8((a, sa), (w, sw), gated=gated, out_dtype=dtype)
        assert_close(f64(got), ref, product_tolerance(ref, gate, dtype), "product")


GROUPED = [
    # counts, alignment of the starts, spare rows at the end
    ([3], 1, 0),
    ([0, 0, 0, 0], 4, 9),
    ([1, 0, 2, 1, 0, 5], 16, 3),
    ([7, 16, 17, 0, 1, 33], 1, 0),
    ([64, 65, 0, 63, 1], 16, 40),
    ([128, 129, 0, 127, 30, 1], 16, 0),
    ([256, 0, 257, 255, 3, 520], 128, 100),
    ([0, 700, 0], 1, 5),
]


@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K,N", [(256, 256), (400, 130), (1040, 514), (7168, 64)])
def test_product_grouped_matches_plain(case, gated, K, N):
    counts, align, spare = GROUPED[case]
    g = torch.Generator(device=DEV).manual_seed(case + K)
    starts, at = [], 0
    for n in counts:
        starts.append(at)
        at += -(-n // align) * align
    say("product grouped", case, gated, K, N)
    check_product(g, at + spare, K, N, counts, starts, gated, torch.bfloat16 if case % 2 else torch.float32)


def test_product_many_groups():
    """As many groups as the layout allows, most of them empty or with one row."""
    g = torch.Generator(device=DEV).manual_seed(11)
    r = np.random.default_rng(11)
    for G, most in ((4096, 2), (1000, 3), (300, 40)):
        counts = r.integers(0, most + 1, G).tolist()
        starts = (np.cumsum(counts) - counts).tolist()
        say("product groups", G)
        check_product(g, max(sum(counts), 1), 64, 48, counts, starts, True, torch.float32)
    # among them large ones, at the ends and in between, so that both kernels have their share
    for G, K, N in ((4096, 64, 64), (1000, 144, 48), (65, 256, 516), (64, 80, 512)):
        counts = r.integers(0, 3, G)
        counts[r.choice(G, min(G, 150), replace=False)] = r.integers(60, 300, min(G, 150))
        counts[0], counts[-1] = 300, 77
        starts = np.cumsum(counts) - counts
        say("product groups, some large", G)
        check_product(g, int(counts.sum()) + 3, K, N, counts.tolist(), starts.tolist(), G % 2 == 0, torch.float32)


def test_product_group_order_and_ranges_outside_the_rows():
    """Groups in any order of rows; ranges that do not exist are empty or cut, and nothing else is written."""
    g = torch.Generator(device=DEV).manual_seed(12)
    for M in (100, 700):
        counts = [20, 30, 5, 10, 10, 1 << 30, -4, 7]
        starts = [60, 0, -3, M, M + 5, M - 15, 40, 1 << 40]
        check_product(g, M, 256, 192, counts, starts, False, torch.float32)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("gated", [False, True])
def test_product_writes_its_rows_alone(dtype, gated):
    """Widths of every remainder: the same as by a product of more channels, and nothing past the end."""
    g = torch.Generator(device=DEV).manual_seed(17)
    K = 64
    for M, widths in ((5, (1, 7, 9, 31, 45)), (2100, (2055, 2061))):  # split, tiles
        a = (codes(g, M, K), torch.rand(M, generator=g, device=DEV))
        for width in widths:
            full = (width + 15) // 16 * 16
            halves = 2 if gated else 1
            w = codes(g, halves, full, K), torch.rand(halves, full, generator=g, device=DEV)
            narrow = tuple(t[:, :width].contiguous().flatten(0, 1) for t in w)
            store = torch.full((M * width + 64,), 9.0, dtype=DTYPES[dtype], device=DEV)
            out = store[:M * width].view(M, width)
            ep.matmul_int8(a, narrow, gated=gated, out=out)
            want = ep.matmul_int8(a, tuple(t.flatten(0, 1) for t in w), gated=gated, out_dtype=DTYPES[dtype])
            assert torch.equal(out, want[:, :width]), (M, width)
            assert (store[M * width:] == 9.0).all()


def test_product_largest_sums():
    """Codes of the largest magnitude over the longest inner size: the sums come near 2^31."""
    g = torch.Generator(device=DEV).manual_seed(13)
    a = torch.full((20, 131056), -128, dtype=torch.int8, device=DEV)
    w = torch.full((36, 131056), -128, dtype=torch.int8, device=DEV)
    w[1] = 127
    one = torch.ones(36, device=DEV)
    out = ep.matmul_int8((a, one[:20].contiguous()), (w, one), out_dtype=torch.float32)
    ref = torch.full((20, 36), 128.0 * 128 * 131056, dtype=torch.float64)
    ref[:, 1] = -128.0 * 127 * 131056
    assert torch.equal(out.cpu(), ref.float())
    check_product(g, 300, 2048, 300, None, None, False, torch.float32, extreme=True)


def test_product_scales_that_are_zero_infinite_or_nan():
    g = torch.Generator(device=DEV).manual_seed(14)
    for M in (5, 300):
        a, w = codes(g, M, 256), codes(g, 64, 256)
        a[1] = 0
        sa = torch.full((M,), 0.01, device=DEV)
        sw = torch.full((64,), 0.01, device=DEV)
        sa[0], sa[2], sw[3] = 0.0, float("nan"), float("nan")
        y = ep.matmul_int8((a, sa), (w, sw), out_dtype=torch.float32)
        bad = torch.isnan(y)
        assert bad[2].all() and bad[:, 3].all() and int(bad.sum()) == 64 + M - 1
        assert (y[0, :3] == 0).all() and (y[1, :3] == 0).all()
        z = ep.matmul_int8((a, sa), (w, sw), gated=True)
        assert torch.isnan(z[2]).all() and torch.isnan(z[:, 3]).all() and int(torch.isnan(z).sum()) == 32 + M - 1
        # gates far below zero close: silu(-large) is -0, not NaN
        y = ep.matmul_int8((torch.full_like(a, 127), torch.full_like(sa, 1e9)),
                           (torch.full_like(w, -127), torch.full_like(sw, 1e9)), gated=True, out_dtype=torch.float32)
        assert (y == 0).all()


# ---------------------------------------------------------------------------- a run of them

def problem(P, S, E, K, H, inter, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T = P * S
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    gate = torch.randn(H, E, generator=g, device=DEV) / H ** 0.5 * 1.5
    up = torch.randn(E, 2 * inter, H, generator=g, device=DEV) / H ** 0.5
    down = torch.randn(E, H, inter, generator=g, device=DEV) / inter ** 0.5

    def channels(w):
        c, s = ep.quantize_int8(w.reshape(-1, w.shape[-1]))
        return c.view(w.shape), s.view(w.shape[:-1])

    return g, x, gate, channels(up), channels(down), torch.randn(E, generator=g, device=DEV) * 0.02


@pytest.mark.parametrize("fixed", [False, True])
def test_expert_rows_are_the_layouts(fixed):
    g = torch.Generator(device=DEV).manual_seed(20)
    P, S, E, K, A = 4, 50, 16, 3, 8
    idx = torch.rand(P * S, E, generator=g, device=DEV).topk(K, 1).indices
    idx[3] = -1
    W = 160 if fixed else 0
    h = ep.get_layout(ep.Config(P, S, 128, K, E, A, num_worst_rows=W), idx)
    start, count = ep.expert_rows(h)
    n = torch.bincount(idx[idx >= 0], minlength=E).cpu().numpy()
    off = h.tensor("expert_offset").cpu().numpy().reshape(P, E // P + 1)
    base = h.tensor("window_row_base").cpu().numpy()
    r, l = np.arange(E) // (E // P), np.arange(E) % (E // P)
    if fixed:
        assert h.status()[1] > 0  # some rows were dropped
        kept = np.clip(np.minimum(n, W - off[r, l]), 0, None)
        np.testing.assert_array_equal(count.cpu().numpy(), kept)
        np.testing.assert_array_equal(start.cpu().numpy()[kept > 0], (base[r] + off[r, l])[kept > 0])
        assert (start.cpu().numpy() <= P * W).all()
    else:
        np.testing.assert_array_equal(count.cpu().numpy(), n)
        np.testing.assert_array_equal(start.cpu().numpy(), base[r] + off[r, l])
    h.free()


def test_route_dispatch_experts_combine():
    """Router, layout, int8 dispatch, gate and up, down, combine: each step against a plain one on what it
    was given, and the experts' rows against the tokens they came from."""
    P, S, E, K, H, inter = 4, 40, 16, 4, 512, 256
    T = P * S
    g, x, gate, up, down, bias = problem(P, S, E, K, H, inter, 21)
    rc = router(E, K, 4, 2, "top2", "sigmoid", scale=2.5)
    logits = x.float() @ gate
    idx, w = check_route(rc, logits, bias)
    h = ep.get_layout(ep.Config(P, S, H, K, E, 16), idx)
    codes_x, scales_x = ep.quantize_int8(x)
    pair = (codes_x.view(torch.uint8), scales_x[:, None].expand(T, H // 128).contiguous())
    rx, rs, rw, meta = ep.dispatch(h, pair, w, scales_col_major=True)
    start, count = ep.expert_rows(h)
    a = (rx.view(torch.int8), rs[0])
    hidden = ep.matmul_int8(a, up, rows=(start, count), gated=True)
    y = ep.matmul_int8(ep.quantize_int8(hidden), down, rows=(start, count))
    out = ep.combine(h, y, w)
    # plain: token by token
    act = ep.quantize_int8(hidden)
    dst = h.tensor("dst_row").cpu().numpy().reshape(T, K)
    xi, xsn = codes_x.cpu().numpy(), scales_x.cpu().numpy()
    hid, yn = f64(hidden), f64(y)
    ai, asn = act[0].cpu().numpy(), act[1].cpu().numpy()
    idn = idx.cpu().numpy()
    upn, upsn, dn, dsn = (t.cpu().numpy() for t in (*up, *down))
    for e in range(E):
        u, j = np.nonzero(idn == e)
        if not len(u):
            continue
        r = dst[u, j]
        ref, gv = plain.product(xi[u], xsn[u], upn[e], upsn[e], True)
        assert_close(hid[r], ref, product_tolerance(ref, gv, torch.bfloat16), ("hidden", e))
        ref, _ = plain.product(ai[r], asn[r], dn[e], dsn[e], False)
        assert_close(yn[r], ref, product_tolerance(ref, None, torch.bfloat16), ("y", e))
    ref = (f64(w)[:, :, None] * yn[dst]).sum(1)
    size = (np.abs(f64(w))[:, :, None] * np.abs(yn[dst])).sum(1)
    assert_close(f64(out), ref, 2.0 ** -8 * np.abs(ref) + (2 * K + 1) * U * size * (1 + 2.0 ** -8), "combine")
    # the gradient of the combine weights flows to the router
    gw = torch.randn(T, K, generator=g, device=DEV)
    dx = ep.route_backward(rc, logits, idx, gw)
    assert torch.isfinite(dx).all() and int((dx != 0).sum()) <= T * K
    h.free()


def serving_step(P, S, E, K, H, inter, seed, worst):
    """Buffers and a function that enqueues one serving step on them, in fixed windows."""
    g, x, gate, up, down, bias = problem(P, S, E, K, H, inter, seed)
    T = P * S
    rc = router(E, K, 4, 2, "top2", "sigmoid", scale=2.5)
    logits = (x.float() @ gate).contiguous()
    idx, w = ep.route(rc, logits, bias=bias)
    h = ep.get_layout(ep.Config(P, S, H, K, E, 16, num_worst_rows=worst), idx)
    R = h.total_rows
    s = dict(x=x, gate=gate, logits=logits, idx=idx, w=w, h=h, g=g, rc=rc)
    s["q"] = (torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV))
    s["scales"] = torch.empty(T, H // 128, device=DEV)
    s["recv"] = (torch.empty(R, H, dtype=torch.uint8, device=DEV), torch.empty(H // 128, R, device=DEV),
                 torch.empty(R, device=DEV), torch.empty(R, 2, dtype=torch.int32, device=DEV))
    s["rows"] = (torch.empty(E, dtype=torch.int64, device=DEV), torch.empty(E, dtype=torch.int32, device=DEV))
    s["hidden"] = torch.zeros(R, inter, dtype=torch.bfloat16, device=DEV)
    s["act"] = (torch.empty(R, inter, dtype=torch.int8, device=DEV), torch.empty(R, device=DEV))
    s["y"] = torch.zeros(R, H, dtype=torch.bfloat16, device=DEV)
    s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    s["grad"] = torch.empty_like(logits)

    def step():
        ep.route(rc, s["logits"], bias=bias, out=(s["idx"], s["w"]))
        ep.relayout(h, s["idx"])
        ep.quantize_int8(s["x"], out=s["q"])
        s["scales"].copy_(s["q"][1][:, None].expand(T, H // 128))
        ep.dispatch(h, (s["q"][0].view(torch.uint8), s["scales"]), s["w"], scales_col_major=True, out=s["recv"])
        ep.expert_rows(h, out=s["rows"])
        a = (s["recv"][0].view(torch.int8), s["recv"][1][0])
        ep.matmul_int8(a, up, rows=s["rows"], gated=True, out=s["hidden"])
        ep.quantize_int8(s["hidden"], out=s["act"])
        ep.matmul_int8(s["act"], down, rows=s["rows"], out=s["y"])
        ep.combine(h, s["y"], s["w"], out=s["out"])
        ep.route_backward(rc, s["logits"], s["idx"], s["w"], out=s["grad"])

    s["step"] = step
    return s


def new_tokens(s, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s["x"].copy_(torch.randn(s["x"].shape, generator=g, device=DEV))
    s["logits"].copy_(s["x"].float() @ s["gate"])


RESULTS = ("idx", "w", "out", "grad")


@pytest.mark.parametrize("S", [1, 33])
def test_captured_step_replays_as_eager(S):
    """The whole step in one graph, replayed on new tokens between eager steps, bit for bit."""
    s = serving_step(4, S, 16, 4, 512, 128, 31, 16 * 16)
    t = serving_step(4, S, 16, 4, 512, 128, 31, 16 * 16)  # the eager twin
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s["step"]()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s["step"]()
    torch.cuda.synchronize()
    for seed in range(4):
        new_tokens(s, seed)
        new_tokens(t, seed)
        graph.replay()
        t["step"]()
        torch.cuda.synchronize()
        for name in RESULTS:
            assert torch.equal(s[name], t[name]), (seed, name)
    s["h"].free()
    t["h"].free()


def test_steps_on_two_streams_at_once():
    """Two steps in flight on two streams share nothing."""
    a = serving_step(4, 64, 16, 4, 512, 256, 41, 16 * 32)
    b = serving_step(4, 48, 16, 4, 512, 256, 42, 16 * 32)
    want = []
    for s in (a, b):
        s["step"]()
        torch.cuda.synchronize()
        want.append([s[n].clone() for n in RESULTS])
        for n in RESULTS:
            s[n].zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s["step"]()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        for n, v in zip(RESULTS, w):
            assert torch.equal(s[n], v), n
        s["h"].free()


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 bytes apart and weights beyond 2^32 bytes: the values of the same
    rows and channels close together."""
    far = 2 ** 31 + 8  # elements between rows
    g = torch.Generator(device=DEV).manual_seed(11)
    near = torch.randn(3, 256, generator=g, device=DEV).bfloat16()
    store = torch.empty(2 * far + 256, dtype=torch.bfloat16, device=DEV)
    apart = store.as_strided((3, 256), (far, 1))
    apart.copy_(near)
    for K in (4, 9):  # several rows a wave, a row a wave
        rc = router(256, K)
        idx, w = ep.route(rc, near)
        got = ep.route(rc, apart)
        assert torch.equal(got[0], idx) and torch.equal(got[1], w)
        gw = torch.randn(3, K, generator=g, device=DEV)
        assert torch.equal(ep.route_backward(rc, apart, idx, gw), ep.route_backward(rc, near, idx, gw))
    for cols in (256, 255):  # read in whole pieces, element by element
        for got, want in zip(ep.quantize_int8(apart[:, :cols]), ep.quantize_int8(near[:, :cols])):
            assert torch.equal(got, want)
    del store, apart
    G, N, K = 3, 65536, 16384  # 3 GiB of weights
    weights = torch.empty(G * N * K, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g).view(G, N, K)
    scales = torch.rand(G, N, generator=g, device=DEV)
    M = 2 ** 18 + 300  # more than 4 GiB of rows, of which the last ones are multiplied
    a = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    a[-300:].random_(-127, 128, generator=g)
    sa = torch.rand(M, generator=g, device=DEV)
    for n in (300, 40):  # by tiles; forty rows alone by the split
        rows = (torch.tensor([0, 0, M - n], device=DEV), torch.tensor([0, 0, n], dtype=torch.int32, device=DEV))
        out = torch.empty(M, 512, dtype=torch.bfloat16, device=DEV)
        tail = weights[:, -512:].contiguous()
        ep.matmul_int8((a, sa), (tail, scales[:, -512:].contiguous()), rows=rows, out=out)
        want = ep.matmul_int8((a[-n:].contiguous(), sa[-n:].contiguous()), (tail[2], scales[2, -512:].contiguous()))
        assert torch.equal(out[-n:], want)
        few = (a[-n:].contiguous(), sa[-n:].contiguous())
        rows = (torch.zeros(3, dtype=torch.int64, device=DEV), torch.tensor([0, 0, n], dtype=torch.int32, device=DEV))
        assert torch.equal(ep.matmul_int8(few, (weights, scales), rows=rows)[:, -512:], want)


def test_bindings_refuse_wrong_tensors():
    rc = router(16, 2)
    x = torch.zeros(4, 16, device=DEV)
    idx = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    a = (torch.zeros(4, 32, dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV))
    b = (torch.zeros(8, 32, dtype=torch.int8, device=DEV), torch.zeros(8, device=DEV))
    for call, error in [
        (lambda: ep.route(rc, x.cpu()), ValueError),
        (lambda: ep.route(rc, x.double()), TypeError),
        (lambda: ep.route(rc, x[:, :8]), ValueError),
        (lambda: ep.route(rc, x.t().contiguous().t()), ValueError),
        (lambda: ep.route(rc, x[:1].expand(4, 16)), ep.EpError),
        (lambda: ep.route(rc, x, bias=torch.zeros(16, dtype=torch.bfloat16, device=DEV)), TypeError),
        (lambda: ep.route(rc, x, bias=torch.zeros(15, device=DEV)), ValueError),
        (lambda: ep.route(rc, x, token_mask=torch.ones(4, dtype=torch.uint8, device=DEV)), TypeError),
        (lambda: ep.route(rc, x, out=(idx.int(), w)), TypeError),
        (lambda: ep.route_backward(rc, x, idx, w.double()), TypeError),
        (lambda: ep.route_backward(rc, x, idx[:3], w), ValueError),
        (lambda: ep.route_backward(rc, x, idx, w, out=x.bfloat16()), TypeError),
        (lambda: ep.quantize_int8(x.int()), TypeError),
        (lambda: ep.quantize_int8(x[0]), ValueError),
        (lambda: ep.quantize_int8(x.t()), ValueError),
        (lambda: ep.matmul_int8(a[0], b), TypeError),
        (lambda: ep.matmul_int8(a, (b[0][:, :16], b[1])), ValueError),
        (lambda: ep.matmul_int8(a, (b[0].view(torch.uint8), b[1])), TypeError),
        (lambda: ep.matmul_int8((a[0], a[1][:3]), b), ValueError),
        (lambda: ep.matmul_int8(a, b, rows=(idx, w)), ValueError),
        (lambda: ep.matmul_int8(a, b, out_dtype=torch.float64), (TypeError, ValueError)),
        (lambda: ep.matmul_int8(a, (b[0][:7], b[1][:7]), gated=True), ValueError),
        (lambda: ep.matmul_int8((a[0][:, :8].contiguous(), a[1]), (b[0][:, :8].contiguous(), b[1])), ep.EpError),
    ]:
        with pytest.raises(error):
            call()
