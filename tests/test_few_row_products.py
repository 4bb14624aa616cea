"""The few-row kernel of the E4M3 and 16-bit products in each of its shapes, dense and by expert, against plain
64-bit implementations; sizes that end inside a step, a row tile and a channel tile.  The shape is asserted, so
that a case stays on it.  Tolerances are those of test_expert_products.py."""

import ctypes
import os

import pytest
import torch

import combine_topk_idx_expert_amd as ep

S = ep.Status

COUNTS = {12: [1, 0, 2, 1, 0, 3], 131: [20, 31, 0, 17, 33, 25], 205: [40, 0, 64, 1, 33, 62], 389: [64, 65, 100, 1, 90, 64]}
# (rows, channels, waves): (rows, bytes of a row, channels before the gate), dense and of six experts
SHAPES = {
    (16, 32, 2): ((12, 400, 258), (12, 400, 258)),
    (16, 32, 4): ((12, 2064, 4098), (12, 2064, 1034)),
    (16, 64, 2): ((12, 400, 8198), (12, 400, 2062)),
    (16, 64, 4): ((12, 2064, 8198), (12, 2064, 2062)),
    (32, 32, 2): ((131, 400, 1034), (205, 400, 518)),
    (32, 32, 4): ((17, 2064, 4100), (205, 4176, 518)),
    (32, 64, 2): ((131, 400, 2062), (389, 400, 518)),
    (32, 64, 4): ((131, 4176, 2062), (205, 2064, 1034)),
    (64, 64, 2): ((131, 400, 4098), (389, 400, 1034)),
    (64, 64, 4): ((131, 2064, 4098), (205, 2064, 2062)),
}


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ep.lib_path()):
        import combine_topk_idx_expert_amd.build as b

        b.build()
    return ep.lib()


def test_shapes_are_named_for_sizes(L):
    for shape, (dense, grouped) in SHAPES.items():
        for gated in (False, True):
            assert ep.debug_split_shape(dense[0], 0, *dense[1:], gated) == shape
            assert ep.debug_split_shape(grouped[0], 6, *grouped[1:], gated) == shape
    assert all(sum(c) + 5 == M for M, c in COUNTS.items())
    # one token, and a decode step of 32 experts whose rows are padded to 16
    assert ep.debug_split_shape(1, 0, 7168, 4096, True) == (16, 32, 4)
    assert ep.debug_split_shape(512, 32, 7168, 4096, True) == (16, 64, 4)
    assert ep.debug_split_shape(8192, 0, 8192, 8192) == ep.debug_split_shape(0, 0, 64, 64) == (0, 0, 0)
    shape = (ctypes.c_int32 * 3)()
    assert L.ep_debug_split_shape(1, 0, 64, 64, 0, None) == S.ERR_NULL
    for inner in (0, -1, 2 * 131056 + 1, (1 << 31) - 1):
        assert L.ep_debug_split_shape(1, 0, inner, 64, 0, shape) == S.ERR_SHAPE
    assert L.ep_debug_split_shape(1, 4096, 2 * 131056, 1 << 20, 0, shape) == S.OK
    assert L.ep_debug_split_shape(1, 0, 64, 63, 1, shape) == S.ERR_SHAPE
    assert L.ep_debug_split_shape(1 << 31, 0, 64, 64, 0, shape) == S.ERR_OVERFLOW


@pytest.fixture(scope="module")
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def layout(t, shape, grouped):
    """(rows, inner bytes, channels, groups, spans, row ranges): groups with nothing between them, and five rows
    behind the last."""
    M, K, N = SHAPES[shape][grouped]
    if not grouped:
        return M, K, N, 0, [(0, M)], None
    count = COUNTS[M]
    start = [sum(count[:i]) for i in range(len(count))]
    return M, K, N, len(count), t.spans(start, count), t.as_rows(start, count)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", list(SHAPES), ids=str)
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_fp8_product_in_every_shape(gpu, shape, grouped, gated):
    import test_expert_products as t

    M, K, N, G, spans, rows = layout(t, shape, grouped)
    assert ep.debug_split_shape(M, G, K, N, gated) == shape
    for dtype, cols in ((torch.bfloat16, False), (torch.float32, True), (torch.float16, True)):
        t.say("few rows", shape, M, K, N, G, gated, dtype, cols)
        a, sa, w, sw = t.fp8_case(M + K, M, K, N, G, gated, cols)
        if G:
            a[-5:] = 0x7F
            (sa.t() if cols else sa)[-5:] = float("nan")
        out = torch.full((M, N // 2 if gated else N), 7.0, dtype=dtype, device=t.DEV)
        ep.matmul_fp8((a, sa), (w, sw), rows=rows, gated=gated, scales_col_major=cols, out=out)
        assert not G or (out[-5:] == 7.0).all()
        x = t.fp8_values(a, sa, cols)
        for e, (s, n) in enumerate(spans):
            if n:
                v = t.fp8_weights(w[e], sw[e], gated) if G else t.fp8_weights(w, sw, gated)
                ref, tol, _, _ = t.expected(x[s:s + n], v, gated, dtype, 0.0 if dtype == torch.float32 else t.DROPPED)
                t.assert_close(out[s:s + n], ref, tol, ("group", e))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", list(SHAPES), ids=str)
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_half_product_in_every_shape(gpu, shape, grouped, gated):
    import test_expert_products as t

    M, K, N, G, spans, rows = layout(t, shape, grouped)
    assert ep.debug_split_shape(M, G, K, N, gated) == shape
    for dtype in (torch.bfloat16, torch.float16):
        t.say("few rows", shape, M, K // 2, N, G, gated, dtype)
        a, w = t.half_case(M + K, M, K // 2, N, G, dtype)
        if G:
            a[-5:] = float("nan")
        out = torch.full((M, N // 2 if gated else N), 7.0, dtype=dtype, device=t.DEV)
        pre = torch.full((M, N), 7.0, dtype=dtype, device=t.DEV) if gated else None
        ep.matmul(a, w, rows=rows, gated=gated, pre=pre, out=out)
        assert not G or ((out[-5:] == 7.0).all() and (pre is None or (pre[-5:] == 7.0).all()))
        for e, (s, n) in enumerate(spans):
            if n:
                ref, tol, y, tol_y = t.expected(t.f64(a[s:s + n]), t.f64(w[e] if G else w), gated, dtype)
                t.assert_close(out[s:s + n], ref, tol, ("group", e))
                if gated:
                    t.assert_close(pre[s:s + n], y, tol_y, ("pre", e))
