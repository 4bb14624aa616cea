"""The norm, its gradient and E4M3 quantising against plain 64-bit implementations.

Tolerances come from the number of roundings; u is half a step of fp32, 2^-24.  Codes and scales of
given rows are single correctly rounded operations and are compared for equality.
"""

import numpy as np
import pytest
import torch

import combine_topk_idx_expert_amd as ep
import plain_expert_layer as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# half of the smallest step above zero
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def say(*a):
    print("[norm]", *a, flush=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def randn(seed, *shape, dtype=torch.float32, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * size).to(dtype)


def assert_close(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    over = np.abs(np.nan_to_num(got) - np.nan_to_num(ref)) - tol
    assert over.max(initial=-1.0) <= 0, (what, over.max(), np.unravel_index(over.argmax(), over.shape))


# The sum of squares has at most 64 additions in a lane, 6 in a wave and 16 among waves; r takes half of
# that relative error and three roundings of its own, y three more.
NORM_ULPS = (64 + 6 + 16) / 2 + 6


def check_norm(x, w, residual=None, eps=EPS, fp8=False):
    y, q, total = ep.rms_norm(x, w, eps=eps, residual=residual, fp8=fp8)
    ref, h = plain.norm(f64(x), f64(w), eps, None if residual is None else f64(residual))
    t = x.dtype
    hs = half_step(t)
    assert y.dtype == t and y.shape == x.shape
    # (h is rounded to fp32 before it is squared: one rounding more)
    assert_close(f64(y), ref, np.nan_to_num((hs + (NORM_ULPS + 2) * U) * np.abs(ref)) + TINY[t], "y")
    if residual is None:
        assert total is None
    else:
        assert_close(f64(total), h, np.nan_to_num((hs + U) * np.abs(h)) + TINY[t], "total")
    if not fp8:
        assert q is None
        return
    codes, scales = q
    amax = np.stack([np.abs(ref[:, b:b + 128]).max(1) for b in range(0, x.shape[1], 128)], 1)
    s = f64(scales)
    assert_close(s, amax / 448, (NORM_ULPS + 4) * U * amax / 448 + 2.0 ** -149, "scales")
    sx = plain.spread(s, x.shape[1])
    # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale below its normal range
    tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sx) * (1 + 2.0 ** -12) + 2 * NORM_ULPS * U * np.abs(ref)
    assert_close(plain.decode(codes.cpu().numpy()) * sx, ref, tol, "codes")


SHAPES = [(1, 7168), (3, 1), (5, 7), (2, 128), (37, 129), (1, 4096), (1025, 512), (1030, 513), (1024, 1000), (1027, 2048),
          (1100, 4096), (300, 2100), (64, 7168), (33, 8192), (9, 8200), (5, 16384), (3, 20000), (2, 32768), (1026, 60)]


@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_norm_matches_plain(N, H, dtype):
    t = DTYPES[dtype]
    for n, (with_residual, w32, fp8) in enumerate([(False, False, False), (True, True, True), (True, False, False),
                                                   (False, True, True)]):
        say(N, H, dtype, with_residual, w32, fp8)
        x = randn(N + H + n, N, H, dtype=t) * (10.0 ** (n - 1))
        x[:, ::17] *= 6
        r = randn(N + H + n + 1, N, H, dtype=t) if with_residual else None
        w = (1 + 0.1 * randn(n, H)).to(torch.float32 if w32 else t)
        check_norm(x, w, r, fp8=fp8)


@pytest.mark.parametrize("H", [128, 777, 4096, 7168])
def test_norm_of_strided_unaligned_and_in_place_rows(H):
    for t in DTYPES.values():
        say("strided", H, t)
        big = randn(H, 40, H + 5, dtype=t)
        x, r = big[:, 3:3 + H], randn(H + 1, 40, 2 * H, dtype=t)[:, H:]
        w = randn(2, H + 1, dtype=t)[1:]
        check_norm(x, w, r, fp8=True)
        xc, rc = x.contiguous(), r.contiguous()
        y, q, total = ep.rms_norm(xc, w, residual=rc, fp8=True)
        xi, ri = xc.clone(), rc.clone()
        y2, q2, total2 = ep.rms_norm(xc, w, residual=ri, fp8=True, keep=False, out=(None, q, ri))
        assert y2 is None and total2 is ri and torch.equal(ri, total)
        ep.rms_norm(xi, w, residual=rc, out=(torch.empty_like(y), None, xi))
        assert torch.equal(xi, total)


def test_norm_rows_at_the_ends_of_fp32():
    """Squares that overflow or vanish, zeros, infinities and NaN: no row disturbs another."""
    for H in (200, 3000, 9000):
        x = randn(7, 1040, H)
        x[0] = 0
        x[1] *= 1e25
        x[2] *= 1e36
        x[3] = 3e38
        x[4] *= 1e-25
        x[5] *= 1e-40
        x[6, 3] = float("inf")
        x[7, 5] = float("nan")
        x[8] = float("-inf")
        x[9, 0] = 3e38
        x[10, 1:] = 0
        x[11] *= 2.0 ** 59
        w = randn(8, H)
        for eps in (1e-6, 1e-30, 1e-44):
            for rows in (1040, 12):
                say("ends", H, eps, rows)
                check_norm(x[:rows], w, eps=eps)
        y, (codes, scales), _ = ep.rms_norm(x[:12], w, fp8=True)
        assert (codes[7] == 0x7F).all() and scales[7].isnan().all()
        assert (codes[8] == 0x7F).all() and scales[6, 0].isnan() and not scales[6, 1:].any()
        assert not (codes[0] & 0x7F).any() and not scales[0].any()
        torch.testing.assert_close(ep.rms_norm(x[12:], w)[0], ep.rms_norm(x, w)[0][12:], rtol=0, atol=0)


def test_codes_of_the_norm_are_those_of_quantising_it():
    for N, H in ((3, 7168), (1300, 1024), (40, 333)):
        x, r, w = randn(1, N, H), randn(2, N, H), randn(3, H)
        y, q, _ = ep.rms_norm(x, w, residual=r, fp8=True)
        codes, scales = ep.quantize_fp8(y)
        assert torch.equal(q[0], codes) and torch.equal(q[1], scales)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("N,H", [(1, 128), (2, 7168), (129, 200), (33, 1), (7, 127), (5, 129), (300, 2048), (3, 50000)])
def test_quantize_matches_plain(N, H, dtype):
    t = DTYPES[dtype]
    x = randn(N * H, N, H + 3, dtype=t)[:, 1:H + 1]
    x = torch.where(randn(1, N, H) > 1.5, 30 * x, x)
    x[0, :: 3] = 0
    for cols in (False, True):
        say("quantise", N, H, dtype, cols)
        codes, scales = ep.quantize_fp8(x, scales_col_major=cols)
        ref, ref_s = plain.quantize_fp8(f64(x))
        np.testing.assert_array_equal(scales.cpu().numpy().T if cols else scales.cpu().numpy(), ref_s)
        np.testing.assert_array_equal(codes.cpu().numpy(), ref)


def test_quantize_blocks_at_the_ends():
    x = randn(4, 24, 384)
    x[0, :128] = 0
    x[1, :128] = -0.0
    x[2, 5], x[2, 200] = float("nan"), float("inf")
    x[3, 5], x[3, 200] = float("-inf"), float("nan")
    x[4] *= 1e-40
    x[5] = 2.0 ** -149
    x[6] = 2.0 ** -149 * 300
    x[7] = 3.4e38
    x[8] *= 2.0 ** -141
    x[9, :] = torch.arange(384, device=DEV) * 2.0 ** -149
    for t in DTYPES.values():
        v = x.to(t)
        codes, scales = ep.quantize_fp8(v)
        ref, ref_s = plain.quantize_fp8(f64(v))
        np.testing.assert_array_equal(scales.cpu().numpy(), ref_s)
        np.testing.assert_array_equal(codes.cpu().numpy(), ref)


def test_quantize_is_what_dispatch_makes():
    P, S, H, K, E = 2, 40, 512, 2, 8
    x = randn(5, P * S, H, dtype=torch.bfloat16)
    x[3, :128] = 0
    x[4, 7] = float("nan")
    x[5, 300] = float("inf")
    h = ep.get_layout(ep.Config(P, S, H, K, E, 4), torch.randint(0, E, (P * S, K), device=DEV))
    w = torch.ones(P * S, K, device=DEV)
    want = ep.dispatch(h, x, w, fp8=True, zero_padding=True)
    got = ep.dispatch(h, ep.quantize_fp8(x), w, zero_padding=True)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b.cpu().numpy())
    h.free()


def check_backward(x, w, g, eps=EPS, through=None):
    gx, gw = ep.rms_norm_backward(x, w, g, eps=eps, grad_total=through)
    ref, ref_w, size, size_w = plain.norm_backward(f64(x), f64(w), f64(g), eps, None if through is None else f64(through))
    t = x.dtype
    assert gx.dtype == t and gw.dtype == torch.float32
    # both sums as in the norm; the mean's error enters with |n| mean |g w n|
    tol = 2 * (NORM_ULPS + 6) * U * size + (half_step(t) + 2 * U) * np.abs(ref) + TINY[t]
    assert_close(f64(gx), ref, tol, "grad_x")
    # a team adds its rows in turn, then up to 1/32 of the 4096 teams and 32 slices are added
    N = x.shape[0]
    chain = min(N, max(4, N / 256) + 1) + 4096 / 32 + 32
    assert_close(f64(gw), ref_w, (NORM_ULPS + 4 + chain) * U * size_w + 2.0 ** -140, "grad_weight")


@pytest.mark.parametrize("N,H", [(0, 64), (1, 1), (1, 7168), (3, 130), (257, 512), (1100, 500), (5000, 512), (900, 1000),
                                 (700, 2048), (2100, 4096), (40, 7168), (5, 8200), (6, 16384), (3, 32768), (12, 20001)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_backward_matches_plain(N, H, dtype):
    t = DTYPES[dtype]
    for w32, with_through in ((False, True), (True, False)):
        say("backward", N, H, dtype, w32, with_through)
        x, g = randn(N + H, N, H, dtype=t) * 3, randn(N + H + 1, N, H, dtype=t)
        w = (1 + 0.1 * randn(1, H)).to(torch.float32 if w32 else t)
        check_backward(x, w, g, through=randn(N, N, H, dtype=t) if with_through else None)


def test_backward_of_strided_rows_in_place_and_again():
    for H in (129, 1024, 7168):
        x, g, p = (randn(s, 50, 2 * H, dtype=torch.bfloat16)[:, H // 2:H // 2 + H] for s in (1, 2, 3))
        w = randn(4, H)
        check_backward(x, w, g, through=p)
        gx, gw = ep.rms_norm_backward(x, w, g, grad_total=p)
        for k in range(2):
            pc, gc = p.contiguous(), g.contiguous()
            ox, ow = ep.rms_norm_backward(x, w, gc, grad_total=pc, out=((pc, gc)[k], torch.empty_like(gw)))
            assert torch.equal(ox, gx) and torch.equal(ow, gw)


def test_backward_rows_at_the_ends_of_fp32():
    for H in (300, 3000):
        x, g, w = randn(1, 8, H), randn(2, 8, H), randn(3, H)
        x[1] *= 1e25
        x[2] *= 1e-25
        x[3] = 0
        x[4] = 3e38
        x[5] *= 1e-40
        for eps in (1e-6, 1e-30, 1e-40):
            # (1e-40: rows of zeros have gradients of 1e20)
            check_backward(x, w, g, eps=eps)


def test_backward_agrees_with_differences():
    """Along random directions, of the 64-bit norm."""
    r = np.random.default_rng(1)
    x, w, g, p = r.standard_normal((6, 300)) * 2, r.standard_normal(300), r.standard_normal((6, 300)), r.standard_normal((6, 300))
    f32 = [torch.from_numpy(v).float().to(DEV) for v in (x, w, g, p)]
    gx, gw = ep.rms_norm_backward(f32[0], f32[1], f32[2], grad_total=f32[3])

    def f(x, w):
        y, h = plain.norm(x, w, EPS)
        return (y * g).sum() + (h * p).sum()

    for k in range(4):
        d, e, step = r.standard_normal(x.shape), r.standard_normal(w.shape), 1e-5
        slope = (f(x + step * d, w + step * e) - f(x - step * d, w - step * e)) / (2 * step)
        got = (f64(gx) * d).sum() + (f64(gw) * e).sum()
        # inputs rounded to fp32 and the third derivative's step^2 are far below this
        assert abs(got - slope) < 1e-4 * (1 + abs(slope))


def test_norm_beyond_32_bits_of_offset():
    N, H = (1 << 32) // 7168 + 700, 7168
    x = torch.zeros(N, H, dtype=torch.bfloat16, device=DEV)
    tail = randn(1, 600, H, dtype=torch.bfloat16)
    x[-600:] = tail
    w = randn(2, H, dtype=torch.bfloat16)
    y, q, total = ep.rms_norm(x, w, residual=x, fp8=True)
    yt, qt, tt = ep.rms_norm(tail, w, residual=tail, fp8=True)
    assert torch.equal(y[-600:], yt) and torch.equal(q[0][-600:], qt[0]) and torch.equal(q[1][-600:], qt[1])
    assert torch.equal(total[-600:], tt)
    codes, scales = ep.quantize_fp8(y)
    ct, st = ep.quantize_fp8(yt)
    assert torch.equal(codes[-600:], ct) and torch.equal(scales[-600:], st)
    del y, total, codes, q
    gx, _ = ep.rms_norm_backward(x, w, x)
    gt, _ = ep.rms_norm_backward(tail, w, tail)
    assert torch.equal(gx[-600:], gt)


def test_norm_on_streams_and_in_graphs():
    x, r, w, g = (randn(k, 300, 2048, dtype=torch.bfloat16) for k in range(4))
    w = w[0].contiguous()

    def step():
        y, q, total = ep.rms_norm(x, w, residual=r, fp8=True)
        return [y, *q, total, *ep.rms_norm_backward(total, w, g, grad_total=y), *ep.quantize_fp8(y)]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(randn(50 + k, 300, 2048, dtype=torch.bfloat16))
        want = [t.clone() for t in step()]
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
