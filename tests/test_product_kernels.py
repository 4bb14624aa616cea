"""Each kernel of the int8 product at the sizes where it can go wrong: every case names the kernel
it is about, and the library has to launch that one for it.

The reference is the product in 64 bits on the device, whose sums stay below 2^53 and are exact.
Tolerances count roundings; u is half a step of fp32, 2^-24.
"""

import ctypes

import numpy as np
import pytest
import torch

import combine_topk_idx_expert_amd as ep

DEV = "cuda:0"
U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# ------------------------------------------------------------------- which kernels run (CPU)

def test_kernels_are_named_for_sizes():
    assert ep.debug_matmul_kernels(0, 0, 64) == ()
    assert ep.debug_matmul_kernels(1, 0, 4096, gated=True) == ("split",)
    for rows in (1, 64):  # few rows, however wide
        assert ep.debug_matmul_kernels(rows, 0, 1 << 20) == ep.debug_matmul_kernels(rows, 0, 1 << 20, True) == ("split",)
    assert ep.debug_matmul_kernels(65, 0, 49152) == ("tiles256",)
    assert ep.debug_matmul_kernels(8192, 0, 8192) == ("tiles256",)
    assert ep.debug_matmul_kernels(1003, 0, 7168) == ("tiles128",)
    assert ep.debug_matmul_kernels(96, 32, 4096, gated=True) == ("split",)
    assert "split" in ep.debug_matmul_kernels(4096 * 40, 4096, 256)


def test_kernel_query_arguments_are_checked():
    f, n = ep.lib().ep_debug_matmul_kernels, ctypes.c_uint32()
    S = ep.Status
    assert f(1, 0, 64, 0, None) == S.ERR_NULL
    for rows, groups, outer, flags, status in [(-1, 0, 64, 0, S.ERR_SHAPE), (1, -1, 64, 0, S.ERR_SHAPE),
                                               (1, 4097, 64, 0, S.ERR_SHAPE), (1, 0, 0, 0, S.ERR_SHAPE),
                                               (1, 0, 63, 1, S.ERR_SHAPE), (1, 0, 64, 2, S.ERR_SHAPE),
                                               (1 << 31, 0, 64, 0, S.ERR_OVERFLOW)]:
        assert f(rows, groups, outer, flags, ctypes.byref(n)) == status


# ------------------------------------------------------------------------------- products

def random_codes(g, *shape):
    return torch.empty(shape, dtype=torch.int8, device=DEV).random_(-128, 128, generator=g)


def extreme_codes(g, *shape):
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, -128, 127).to(torch.int8)


def reference(a, sa, w, sw, gated):
    """One group in 64 bits, and the bound's relative part without the output's rounding: three roundings
    of a value; a gate's silu is off by those times 1 + |gate| and by a few more."""
    y = a.double() @ w.double().t().contiguous() * sa.double()[:, None] * sw.double()[None, :]
    if not gated:
        return y, torch.full_like(y, 3.1 * U)
    half = y.shape[1] // 2
    gate = y[:, :half]
    return gate / (1 + torch.exp(-gate)) * y[:, half:], (4 * (1 + gate.abs()) + 16) * U


def check(kernels, M, K, width, counts=None, starts=None, gated=False, dtype=torch.float32, make=random_codes, seed=0,
          spoil=None):
    """One product against the reference; rows of no group keep what they held."""
    G = 0 if counts is None else len(counts)
    N = width * (2 if gated else 1)
    assert ep.debug_matmul_kernels(M, G, N, gated) == kernels
    g = torch.Generator(device=DEV).manual_seed(seed + M + K + width)
    a = make(g, M, K)
    w = make(g, *((G, N, K) if G else (N, K)))
    sa = (torch.rand(M, generator=g, device=DEV) + 0.5) * 2.0 ** -7
    sw = (torch.rand(w.shape[:-1], generator=g, device=DEV) + 0.5) * 2.0 ** -7 / K ** 0.5
    if spoil:
        spoil(sa, sw)
    out = torch.full((M, width), -77.0, dtype=dtype, device=DEV)
    rows = None
    if G:
        rows = (torch.tensor(starts, dtype=torch.int64, device=DEV), torch.tensor(counts, dtype=torch.int32, device=DEV))
    ep.matmul_int8((a, sa), (w, sw), rows=rows, gated=gated, out=out)
    written = torch.zeros(M, dtype=torch.bool, device=DEV)
    half = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    for e in range(max(G, 1)):
        lo, n = (starts[e], counts[e]) if G else (0, M)
        if n <= 0 or lo < 0 or lo >= M:
            continue
        hi = min(lo + n, M)
        written[lo:hi] = True
        ref, rel = reference(a[lo:hi], sa[lo:hi], w[e] if G else w, sw[e] if G else sw, gated)
        got = out[lo:hi].double()
        tol = ref.abs() * (rel + half * (1 + rel)) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -148)
        bad = torch.isnan(ref)
        assert torch.equal(torch.isnan(got), bad), e
        over = torch.where(bad, -1.0, (got - ref).abs() - tol)
        assert over.max() <= 0, (e, float(over.max()), divmod(int(over.argmax()), width))
    assert (out[~written] == -77.0).all()
    return out


def laid_out(counts, align):
    starts, at = [], 0
    for n in counts:
        starts.append(at)
        at += -(-n // align) * align
    return starts, at


T128, T256, BOTH128, BOTH256 = ("tiles128",), ("tiles256",), ("split", "tiles128"), ("split", "tiles256")

DENSE = [
    # kernel, rows, inner, columns of out for a plain and a gated product
    (T128, 300, 256, 8192, 4096), (T128, 129, 400, 12037, 6021), (T128, 1003, 2048, 7168, 2000), (T128, 1025, 144, 3000, 1500),
    (T128, 641, 16, 4100, 2050), (T128, 300, 1040, 8195, 4101), (T128, 127, 80, 24577, 12300),
    (T256, 300, 1040, 24577, 12289), (T256, 2100, 256, 5637, 2821), (T256, 4096 + 1, 656, 3000, 1500),
    (T256, 4096 + 129, 2064, 2817, 1409), (T256, 65, 160, 49151, 24577), (T256, 513, 16, 16300, 8200),
    (T256, 6000, 7168, 2100, 1100), (T256, 1025, 80, 10000, 4993),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(DENSE)))
@pytest.mark.parametrize("gated", [False, True])
def test_dense_tiles_match(gpu, case, gated):
    kernels, M, K, plain, half = DENSE[case]
    for dtype in (torch.bfloat16, torch.float32) if case % 3 else DTYPES.values():
        print("[product] dense", M, K, gated, dtype, flush=True)
        check(kernels, M, K, half if gated else plain, gated=gated, dtype=dtype)


GROUPED = [
    # kernels, counts, alignment of the starts, spare rows, columns of out for a plain and a gated product
    (BOTH128, [128, 129, 0, 127, 30, 1], 16, 0, 5615, 2805),
    (BOTH256, [128, 129, 0, 127, 30, 1], 16, 0, 7600, 3717),
    (BOTH128, [64, 65, 0, 63, 1, 200], 16, 40, 4865, 2430),
    (BOTH256, [64, 65, 0, 63, 1, 200], 1, 40, 7190, 3590),
    (T128, [256, 0, 257, 255, 3, 520], 128, 100, 2100, 1025),
    (T256, [256, 0, 257, 255, 3, 520], 128, 100, 4090, 2043),
    (BOTH256, [0, 700, 0], 1, 5, 9733, 4869),
    (BOTH128, [0, 700, 0], 1, 5, 5110, 2550),
    (BOTH128, [513] + [0] * 5 + [66] * 4 + [3] * 2, 1, 700, 2040, 1020),
    (BOTH256, [0] * 40 + [513] + [65] * 20 + [1] * 3, 16, 900, 1024, 500),
    (BOTH256, [90] * 200 + [64] * 100, 1, 0, 130, 70),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [16, 400, 1040, 7168])
def test_grouped_tiles_match(gpu, case, gated, K):
    kernels, counts, align, spare, plain, half = GROUPED[case]
    starts, at = laid_out(counts, align)
    if len(counts) * plain * K > 3 << 30:
        K = 2064
    print("[product] grouped", case, gated, K, flush=True)
    check(kernels, at + spare, K, half if gated else plain, counts, starts, gated,
          (torch.bfloat16, torch.float32, torch.float16)[case % 3])


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kernels,M,width", [(BOTH128, 700, 3300), (BOTH256, 700, 6000), (T128, 2500, 1500), (T256, 2500, 3000)])
def test_tiles_of_ranges_outside_the_rows_and_out_of_order(gpu, kernels, M, width, gated):
    """Groups in any order of rows; ranges that do not exist are empty or cut, and nothing else is written."""
    big = M // 5
    counts = [big, 90, 70, 1 << 30, 300, 80, -4, 200, 66]
    starts = [M - 130 - big, 0, -3, M - 120, M + 5, 120, 40, 1 << 40, M]
    check(kernels, M, 272, width // 2 if gated else width, counts, starts, gated)


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kernels,M,width", [(("split",), 5, 64), (T128, 300, 8192), (T256, 300, 24577)])
def test_scales_that_are_zero_infinite_or_nan(gpu, kernels, M, width, gated):
    """Rows and channels whose scales are NaN are NaN, and no other."""
    width = width // 2 if gated else width

    def spoil(sa, sw):
        sa[0], sa[2], sa[M - 1] = 0.0, float("nan"), float("nan")
        sw[3], sw[width - 1] = float("nan"), float("nan")

    out = check(kernels, M, 256, width, gated=gated, spoil=spoil)
    assert torch.isnan(out[2]).all() and torch.isnan(out[M - 1]).all()
    assert torch.isnan(out[:, 3]).all() and torch.isnan(out[:, width - 1]).all()
    assert int(torch.isnan(out).sum()) == 2 * width + 2 * M - 4


@pytest.mark.gpu
@pytest.mark.parametrize("kernels,M,K,width", [(T128, 300, 2048, 8200), (T256, 300, 2048, 24577), (T256, 300, 131056, 24577)])
def test_largest_codes_by_tiles(gpu, kernels, M, K, width):
    """Codes of the largest magnitude: long sums come near 2^31 (and stay exact)."""
    if K < 100000:
        check(kernels, M, K, width, make=extreme_codes)
        return
    assert ep.debug_matmul_kernels(M, 0, width) == kernels
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((width, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    out = ep.matmul_int8((a, torch.ones(M, device=DEV)), (w, torch.ones(width, device=DEV)), out_dtype=torch.float32)
    assert (out[:, 0::2] == float(np.float32(128.0 * 128 * K))).all()
    assert (out[:, 1::2] == float(np.float32(-128.0 * 127 * K))).all()


@pytest.mark.gpu
def test_rows_and_weights_beyond_32_bits(gpu):
    """Rows and weights of the last groups start more than 2^32 bytes in: by tiles and, forty rows of one group,
    by the split, the values of the same rows and weights close together."""
    g = torch.Generator(device=DEV).manual_seed(11)
    G, N, K, M = 1100, 256, 16384, 2 ** 18 + 340
    assert ep.debug_matmul_kernels(M, G, N) == BOTH256 and (G - 2) * N * K > 2 ** 32 and (M - 340) * K >= 2 ** 32
    a = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    a[-340:].random_(-127, 128, generator=g)
    w = torch.zeros(G, N, K, dtype=torch.int8, device=DEV)
    w[-2:].random_(-127, 128, generator=g)
    sa, sw = torch.rand(M, generator=g, device=DEV), torch.rand(G, N, generator=g, device=DEV)
    start = torch.zeros(G, dtype=torch.int64, device=DEV)
    count = torch.zeros(G, dtype=torch.int32, device=DEV)
    start[-2], count[-2] = M - 340, 40
    start[-1], count[-1] = M - 300, 300
    out = ep.matmul_int8((a, sa), (w, sw), rows=(start, count))
    for e, lo, hi in ((G - 2, M - 340, M - 300), (G - 1, M - 300, M)):
        want = ep.matmul_int8((a[lo:hi].contiguous(), sa[lo:hi].contiguous()), (w[e], sw[e]))
        assert torch.equal(out[lo:hi], want), e


@pytest.mark.gpu
def test_one_row_a_wave_of_rows_beyond_32_bits(gpu):
    """The routers of more than 16 choices, and of more than 1024 experts, on rows more than 2^32 bytes apart."""
    g = torch.Generator(device=DEV).manual_seed(12)
    far = 2 ** 31 + 8  # elements between rows
    store = torch.empty(2 * far + 1100, dtype=torch.bfloat16, device=DEV)
    for E, K in ((256, 17), (1030, 5)):
        near = torch.randn(3, E, generator=g, device=DEV).bfloat16()
        apart = store.as_strided((3, E), (far, 1))
        apart.copy_(near)
        for renorm in (True, False):
            rc = ep.RouteConfig(E=E, K=K, renormalize=renorm)
            idx, w = ep.route(rc, near)
            got = ep.route(rc, apart)
            assert torch.equal(got[0], idx) and torch.equal(got[1], w)
            gw = torch.randn(3, K, generator=g, device=DEV)
            assert torch.equal(ep.route_backward(rc, apart, idx, gw), ep.route_backward(rc, near, idx, gw))
