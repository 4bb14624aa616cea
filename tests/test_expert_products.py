"""E4M3 and 16-bit products against plain 64-bit implementations.

Tolerances: u is half a step of fp32, 2^-24.  A sum of K products is off by at most K additions of 2 u each
(a matrix instruction may cut instead of rounding) relative to the sum of the magnitudes; block scales add
a product for each block.  The result is rounded once to its type.  For 16-bit results of E4M3 rows
the matrix instruction drops what lies 2^-14 and more below the largest of up to 16 products, of each of
them: at most 16 * 2^-14 = 2^-10 of the sum of the magnitudes.
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
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def say(*a):
    print("[products]", *a, flush=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# a value from here on rounds to an infinity
LARGEST = {t: torch.finfo(t).max * (1 + torch.finfo(t).eps / 4) for t in DTYPES.values()}


def assert_close(got, ref, tol, what):
    dtype, got = got.dtype, f64(got)
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    # a value that may round past its type's largest is an infinity of its sign
    past = np.isinf(got) & (np.abs(ref) + tol >= LARGEST[dtype]) & (np.sign(got) == np.sign(ref))
    got = np.where(past, ref, got)
    over = np.abs(np.nan_to_num(got) - np.nan_to_num(ref)) - tol
    assert over.max(initial=-1.0) <= 0, (what, over.max(), np.unravel_index(over.argmax(), over.shape))


def times(a, b, t):
    """a @ b.T and |a| @ |b|.T in 64 bits, on the GPU."""
    a, b = torch.from_numpy(a).to(DEV), torch.from_numpy(b).to(DEV)
    return (a @ b.t()).cpu().numpy(), (a.abs() @ b.abs().t()).cpu().numpy()


DROPPED = 2.0 ** -10


def expected(a, w, gated, dtype, dropped=0.0):
    """(result, tolerance, product before the gate, its tolerance) of float64 operands."""
    y, size = times(a, w, dtype)
    off = ((2 * a.shape[1] + 16) * U + dropped) * size
    hs = torch.finfo(dtype).eps / 2
    tol_y = off + (hs + U) * np.abs(y) + TINY[dtype]
    if not gated:
        return y, tol_y, y, tol_y
    half = y.shape[1] // 2
    g, u = y[:, :half], y[:, half:]
    ref = plain.gate(y)
    # the gate's slope is at most 1.1; silu itself: 2^-16 for 16-bit results, some roundings for fp32
    own = 2.0 ** -16 if dtype != torch.float32 else 16 * U
    # (fp32: the exponential's argument, rounded, is off by |g| u)
    own = own + (np.minimum(np.abs(g), 110) * 2 * U if dtype == torch.float32 else 0)
    tol = 1.1 * off[:, :half] * (np.abs(u) + off[:, half:]) + np.abs(plain.silu(g)) * off[:, half:]
    return ref, tol + (hs + U + own) * np.abs(ref) + TINY[dtype], y, tol_y


def groups_of(counts, align=16, gap=0):
    n = np.asarray(counts)
    start = np.concatenate([[0], np.cumsum((n + align - 1) // align * align + gap)])[:-1]
    M = int((start + n).max(initial=0)) + 5
    return start, n, M


def as_rows(start, count):
    return (torch.from_numpy(np.asarray(start, np.int64)).to(DEV), torch.from_numpy(np.asarray(count, np.int32)).to(DEV))


# ------------------------------------------------------------------------------------ E4M3

def codes(seed, *shape):
    g = gen(seed)
    return (torch.randn(shape, generator=g, device=DEV) * 60).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def fp8_case(seed, M, K, N, G, gated, cols):
    g = gen(seed + 1)
    kb, width = plain.blocks(K), N // 2 if gated else N
    nb = 2 * plain.blocks(width) if gated else plain.blocks(N)
    a, w = codes(seed, M, K), codes(seed + 2, *((G, N, K) if G else (N, K)))
    sa = torch.exp(torch.randn((kb, M) if cols else (M, kb), generator=g, device=DEV)) / 50
    sw = torch.exp(torch.randn(((G, nb, kb) if G else (nb, kb)), generator=g, device=DEV)) / 50 / K ** 0.5
    return a, sa, w, sw


def fp8_values(a, sa, cols):
    s = sa.cpu().numpy().T if cols else sa.cpu().numpy()
    return plain.decode(a.cpu().numpy()) * plain.spread(s, a.shape[1])


def fp8_weights(w, sw, gated):
    return plain.decode(w.cpu().numpy()) * plain.weight_scales(sw.cpu().numpy(), *w.shape, gated)


def check_fp8_dense(M, K, N, gated, dtype, cols, seed=0):
    a, sa, w, sw = fp8_case(seed, M, K, N, 0, gated, cols)
    got = ep.matmul_fp8((a, sa), (w, sw), gated=gated, scales_col_major=cols, out_dtype=dtype)
    ref, tol, _, _ = expected(fp8_values(a, sa, cols), fp8_weights(w, sw, gated), gated, dtype,
                              0.0 if dtype == torch.float32 else DROPPED)
    assert got.dtype == dtype
    assert_close(got, ref, tol, "fp8 product")


DENSE = [(1, 128, 16), (1, 7168, 512), (1, 16, 2), (3, 48, 34), (17, 144, 258), (33, 272, 130), (64, 1024, 640), (65, 128, 96),
         (130, 400, 1026), (200, 2064, 260), (512, 512, 512), (700, 640, 3900), (1003, 256, 7168), (2100, 1168, 6150),
         (4096, 384, 4096), (4100, 16, 3330)]


@pytest.mark.parametrize("M,K,N", DENSE)
@pytest.mark.parametrize("gated", [False, True])
def test_fp8_dense_matches_plain(M, K, N, gated):
    for n, (dtype, cols) in enumerate([("bf16", False), ("fp32", True), ("fp16", True)]):
        say("fp8", M, K, N, gated, dtype, cols, ep.debug_matmul_kernels(M, 0, N, gated))
        check_fp8_dense(M, K, N, gated, DTYPES[dtype], cols, seed=n)


GROUPS = [
    # counts, inner, outer
    ([3, 0, 2, 1], 256, 96),
    ([0, 0, 0], 128, 64),
    ([1], 144, 130),
    ([17, 64, 65, 0, 130, 5], 1040, 514),
    ([128, 129, 255, 256, 257, 300], 272, 1300),
    ([700, 1, 0, 520, 64, 900, 33], 640, 2306),
    (list(range(0, 70)), 80, 36),
    ([2000, 3000, 0, 1500, 20], 528, 4100),
]


def spans(start, count):
    return [(int(s), int(n)) for s, n in zip(start, count)]


@pytest.mark.parametrize("counts,K,N", GROUPS, ids=[str(i) for i in range(len(GROUPS))])
@pytest.mark.parametrize("gated", [False, True])
def test_fp8_groups_match_plain(counts, K, N, gated):
    start, count, M = groups_of(counts, gap=3)
    G = len(counts)
    for dtype, cols in (("bf16", True), ("fp32", False)):
        say("fp8 groups", len(counts), K, N, gated, dtype, cols, ep.debug_matmul_kernels(M, G, N, gated))
        t = DTYPES[dtype]
        a, sa, w, sw = fp8_case(len(counts), M, K, N, G, gated, cols)
        # what lies between the groups is NaN: it may not reach any row
        between = torch.ones(M, dtype=torch.bool, device=DEV)
        for s, n in spans(start, count):
            between[s:s + n] = False
        a[between] = 0x7F
        (sa.t() if cols else sa)[between] = float("nan")
        width = N // 2 if gated else N
        out = torch.full((M, width), 7.0, dtype=t, device=DEV)
        ep.matmul_fp8((a, sa), (w, sw), rows=as_rows(start, count), gated=gated, scales_col_major=cols, out=out)
        assert (out[between] == 7.0).all()
        x = fp8_values(a, sa, cols)
        for e, (s, n) in enumerate(spans(start, count)):
            if n:
                ref, tol, _, _ = expected(x[s:s + n], fp8_weights(w[e], sw[e], gated), gated, t,
                                          0.0 if t == torch.float32 else DROPPED)
                assert_close(out[s:s + n], ref, tol, ("group", e))


@pytest.mark.parametrize("M,K,N", [(2, 144, 64), (130, 144, 64), (2100, 272, 6150), (4096, 272, 4096)])
def test_fp8_nan_codes_stay_in_their_row_and_channel(M, K, N):
    """The inner size ends inside a block, and what follows a row or channel is the next one's codes."""
    a, sa, w, sw = fp8_case(9, M, K, N, 0, False, False)
    a[1, 0] = 0x7F
    w[5, 3] = 0xFF
    got = ep.matmul_fp8((a, sa), (w, sw), out_dtype=torch.float32)
    nan = got.isnan()
    want = torch.zeros_like(nan)
    want[1], want[:, 5] = True, True
    assert torch.equal(nan, want)


def test_fp8_takes_torch_float8_and_scales_at_the_ends():
    a, sa, w, sw = fp8_case(3, 70, 512, 256, 0, False, False)
    want = ep.matmul_fp8((a, sa), (w, sw))
    got = ep.matmul_fp8((a.view(torch.float8_e4m3fn), sa), (w.view(torch.float8_e4m3fn), sw))
    assert torch.equal(got, want)
    sa[4] = 0
    sa[5, 1] = float("inf")
    sa[6, 2] = float("nan")
    got = ep.matmul_fp8((a, sa), (w, sw))
    assert (got[4] == 0).all() and not got[5].isfinite().any() and got[6].isnan().all()
    keep = torch.ones(70, dtype=torch.bool, device=DEV)
    keep[4:7] = False
    assert torch.equal(got[keep], want[keep])


# ----------------------------------------------------------------------------------- 16 bit

def half_case(seed, M, K, N, G, dtype):
    g = gen(seed)
    a = torch.randn((M, K), generator=g, device=DEV).to(dtype)
    w = (torch.randn((G, N, K) if G else (N, K), generator=g, device=DEV) / K ** 0.5).to(dtype)
    return a, w


HALF = [(1, 64, 16), (1, 7168, 512), (1, 8, 2), (3, 24, 34), (17, 72, 258), (33, 136, 130), (64, 1024, 640), (65, 128, 96),
        (130, 200, 1026), (200, 1032, 260), (512, 512, 512), (700, 320, 3900), (1003, 256, 7168), (2100, 584, 6150),
        (4096, 192, 4096), (4100, 8, 3330)]


@pytest.mark.parametrize("M,K,N", HALF)
@pytest.mark.parametrize("gated", [False, True])
def test_half_dense_matches_plain(M, K, N, gated):
    for dtype in (torch.bfloat16, torch.float16):
        say("half", M, K, N, gated, dtype, ep.debug_matmul_kernels(M, 0, N, gated))
        a, w = half_case(M + K, M, K, N, 0, dtype)
        pre = torch.empty(M, N, dtype=dtype, device=DEV) if gated else None
        got = ep.matmul(a, w, gated=gated, pre=pre)
        ref, tol, y, tol_y = expected(f64(a), f64(w), gated, dtype)
        assert got.dtype == dtype
        assert_close(got, ref, tol, "product")
        if gated:
            assert_close(pre, y, tol_y, "pre")
            assert torch.equal(ep.matmul(a, w, gated=True), got)


@pytest.mark.parametrize("counts,K,N", [(c, k // 16 * 8, n) for c, k, n in GROUPS], ids=[str(i) for i in range(len(GROUPS))])
@pytest.mark.parametrize("gated", [False, True])
def test_half_groups_match_plain(counts, K, N, gated):
    start, count, M = groups_of(counts, gap=3)
    G = len(counts)
    for dtype in (torch.bfloat16, torch.float16):
        say("half groups", len(counts), K, N, gated, dtype, ep.debug_matmul_kernels(M, G, N, gated))
        a, w = half_case(G, M, K, N, G, dtype)
        between = torch.ones(M, dtype=torch.bool, device=DEV)
        for s, n in spans(start, count):
            between[s:s + n] = False
        a[between] = float("nan")
        out = torch.full((M, N // 2 if gated else N), 7.0, dtype=dtype, device=DEV)
        pre = torch.full((M, N), 7.0, dtype=dtype, device=DEV) if gated else None
        ep.matmul(a, w, rows=as_rows(start, count), gated=gated, pre=pre, out=out)
        assert (out[between] == 7.0).all() and (not gated or (pre[between] == 7.0).all())
        for e, (s, n) in enumerate(spans(start, count)):
            if n:
                ref, tol, y, tol_y = expected(f64(a[s:s + n]), f64(w[e]), gated, dtype)
                assert_close(out[s:s + n], ref, tol, ("group", e))
                if gated:
                    assert_close(pre[s:s + n], y, tol_y, ("pre", e))


@pytest.mark.parametrize("M,K,N", [(2, 72, 64), (130, 72, 64), (2100, 136, 6150), (4096, 136, 4096)])
def test_half_nan_and_infinite_values_stay_in_their_row_and_channel(M, K, N):
    a, w = half_case(9, M, K, N, 0, torch.bfloat16)
    a[1, 0] = float("nan")
    w[5, 3] = float("inf")
    w[7, 0] = float("nan")
    got = ep.matmul(a, w)
    bad = ~got.isfinite()
    want = torch.zeros_like(bad)
    want[1], want[:, 5], want[:, 7] = True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("M,K,N", [(4100, 128, 3330), (4100, 256, 3330), (4100, 384, 3330)])
@pytest.mark.parametrize("gated", [False, True])
def test_short_inner_sizes_over_many_tiles(M, K, N, gated):
    """One, two and three steps a tile, more tiles than workgroups."""
    check_fp8_dense(M, K, N, gated, torch.bfloat16, True)
    a, w = half_case(1, M, K // 2, N, 0, torch.bfloat16)
    ref, tol, _, _ = expected(f64(a), f64(w), gated, torch.bfloat16)
    assert_close(ep.matmul(a, w, gated=gated), ref, tol, "product")


@pytest.mark.parametrize("op", ["fp8", "half"])
def test_as_many_groups_as_experts_may_be(op):
    G, K, N = 4096, 32, 24
    count = np.random.default_rng(1).integers(0, 4, G)
    count[7], count[4000] = 300, 170
    start, count, M = groups_of(count)
    rows = as_rows(start, count)
    if op == "fp8":
        a, sa, w, sw = fp8_case(1, M, K, N, G, True, False)
        got = ep.matmul_fp8((a, sa), (w, sw), rows=rows, gated=True, out_dtype=torch.float32)
        x, v, dropped, t = fp8_values(a, sa, False), lambda e: fp8_weights(w[e], sw[e], True), 0.0, torch.float32
    else:
        a, w = half_case(1, M, K, N, G, torch.bfloat16)
        got = ep.matmul(a, w, rows=rows, gated=True)
        x, v, dropped, t = f64(a), lambda e: f64(w[e]), 0.0, torch.bfloat16
    for e, (s, n) in enumerate(spans(start, count)):
        if n:
            ref, tol, _, _ = expected(x[s:s + n], v(e), True, t, dropped)
            assert_close(got[s:s + n], ref, tol, ("group", e))


@pytest.mark.parametrize("op", ["fp8", "half"])
def test_ranges_outside_the_rows_are_cut(op):
    """Row ranges come from the device: those past the rows are cut, those that start outside are empty."""
    M, K, N = 300, 128, 96
    start, count = [-3, 290, 300, 1 << 40, 0, 100, 64], [5, 100, 4, 9, 40, -2, 0]
    rows = as_rows(start, count)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    G = len(start)
    if op == "fp8":
        a, sa, w, sw = fp8_case(1, M, K, N, G, False, False)
        ep.matmul_fp8((a, sa), (w, sw), rows=rows, out=out)
        one = lambda e, s, n: ep.matmul_fp8((a[s:s + n], sa[s:s + n]), (w[e], sw[e]))
    else:
        a, w = half_case(1, M, K, N, G, torch.bfloat16)
        ep.matmul(a, w, rows=rows, out=out)
        one = lambda e, s, n: ep.matmul(a[s:s + n], w[e])
    touched = torch.zeros(M, dtype=torch.bool, device=DEV)
    for e, s, n in ((1, 290, 10), (4, 0, 40)):
        touched[s:s + n] = True
        torch.testing.assert_close(out[s:s + n], one(e, s, n), rtol=2 ** -7, atol=1e-3)
    assert (out[~touched] == 7.0).all()


@pytest.mark.parametrize("op", ["fp8", "half"])
def test_more_than_32_bits_of_offset(op):
    M, K = (1 << 32) // 4096 + 300, 4096
    if op == "fp8":
        a = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
        a[-300:] = codes(1, 300, K)
        sa = torch.ones(M, K // 128, device=DEV) / 64
        w, sw = codes(2, 2, 256, K), torch.ones(2, 2, K // 128, device=DEV) / 64
        run = lambda x, s, r: ep.matmul_fp8((x, s), (w, sw), rows=r)
    else:
        a = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
        a[-300:] = torch.randn(300, K, generator=gen(1), device=DEV)
        sa = a
        w = torch.randn(2, 256, K, generator=gen(2), device=DEV).to(torch.bfloat16)
        run = lambda x, s, r: ep.matmul(x, w, rows=r)
    out = run(a, sa, as_rows([0, M - 300], [200, 300]))
    want = run(a[-300:].contiguous(), sa[-300:].contiguous(), as_rows([0, 0], [0, 300]))
    torch.testing.assert_close(out[-300:], want, rtol=2 ** -6, atol=1e-2)
