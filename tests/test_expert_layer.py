"""The expert layer as it is used: norm, router, layout, dispatch, products, combine, and back.

Each stage is compared with the plain 64-bit implementation of what the stage before gave, with the
tolerances of the operators' own tests."""

import numpy as np
import pytest
import torch

import combine_topk_idx_expert_amd as ep
import plain_expert_layer as plain
from test_expert_gradients import close_product, product_gradient
from test_expert_products import (DEV, DROPPED, TINY, U, as_rows, assert_close, expected, f64, fp8_values, fp8_weights, gen,
                                  spans)
from test_norm import check_norm

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


P, S, H, F, K, E = 2, 96, 256, 192, 3, 16
T = P * S


def randn(seed, *shape, dtype=BF16, size=1.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * size).to(dtype)


def layout(idx, worst=0):
    return ep.get_layout(ep.Config(P, S, H, K, E, 16, num_worst_rows=worst), idx)


def weight_pair(seed, outer, inner, gated):
    """E4M3 weights of all experts with scales for 128 x 128, made once, as a checkpoint holds them."""
    w = randn(seed, E, outer, inner, dtype=torch.float32, size=inner ** -0.5)
    halves = w.chunk(2, 1) if gated else (w,)
    codes, scales = [], []
    for h in halves:
        n = h.shape[1]
        pad = torch.nn.functional.pad(h, (0, -inner % 128, 0, -n % 128))
        b = pad.view(E, pad.shape[1] // 128, 128, pad.shape[2] // 128, 128)
        s = b.abs().amax((2, 4)) / 448
        q = (b / s[:, :, None, :, None]).view(pad.shape)[:, :n, :inner]
        codes.append(q.to(torch.float8_e4m3fn))
        scales.append(s)
    return torch.cat([c.view(torch.uint8) for c in codes], 1).contiguous(), torch.cat(scales, 1).contiguous()


@pytest.mark.parametrize("col_major", [False, True])
def test_fp8_serving_layer(col_major):
    x, res, wn, router = randn(1, T, H), randn(2, T, H), 1 + 0.1 * randn(3, H, dtype=torch.float32), randn(4, E, H)
    gate_up, down = weight_pair(5, 2 * F, H, True), weight_pair(6, H, F, False)
    y, q, total = ep.rms_norm(x, wn, residual=res, fp8=True)
    check_norm(x, wn, res, fp8=True)
    idx, w = ep.route(ep.RouteConfig(E=E, K=K), ep.matmul(y, router))
    h = layout(idx)
    rx, rs, _, _ = ep.dispatch(h, q, w, zero_padding=True, scales_col_major=col_major)
    rows = ep.expert_rows(h)
    act = ep.matmul_fp8((rx, rs), gate_up, rows=rows, gated=True, scales_col_major=col_major,
                        out=torch.zeros(h.total_rows, F, dtype=BF16, device=DEV))
    aq = ep.quantize_fp8(act, scales_col_major=col_major)
    out = ep.matmul_fp8(aq, down, rows=rows, scales_col_major=col_major,
                        out=torch.zeros(h.total_rows, H, dtype=BF16, device=DEV))
    combined = ep.combine(h, out, w, bias=total)
    xv, av = fp8_values(rx, rs, col_major), fp8_values(aq[0], aq[1], col_major)
    start, count = (t.tolist() for t in rows)
    assert sum(count) == T * K
    for e, (s, n) in enumerate(spans(start, count)):
        if n:
            ref, tol, _, _ = expected(xv[s:s + n], fp8_weights(gate_up[0][e], gate_up[1][e], True), True, BF16, DROPPED)
            assert_close(act[s:s + n], ref, tol, ("gate up", e))
            ref, tol, _, _ = expected(av[s:s + n], fp8_weights(down[0][e], down[1][e], False), False, BF16, DROPPED)
            assert_close(out[s:s + n], ref, tol, ("down", e))
    # combine adds the choices in order in fp32, rounds once; the codes stand in the rows it names
    dst = h.tensor("dst_row").view(T, K).cpu().numpy()
    ref = (f64(out)[dst] * f64(w)[:, :, None]).sum(1) + f64(total)
    size = (np.abs(f64(out))[dst] * f64(w)[:, :, None]).sum(1) + np.abs(f64(total))
    # (bf16 keeps 8 bits: a step is 2^-7 of a value just above a power of two, half of it 2^-8)
    assert_close(combined, ref, torch.finfo(BF16).eps / 2 * np.abs(ref) + 8 * U * size, "combine")
    h.free()


def training_step(x, res, wn, router, gate_up, down, grad_out, worst=0):
    """Forward and backward pass; everything that the stages make, by name."""
    v = {}
    v["y"], _, v["total"] = ep.rms_norm(x, wn, residual=res)
    logits = ep.matmul(v["y"], router)
    rc = ep.RouteConfig(E=E, K=K)
    v["idx"], v["w"] = ep.route(rc, logits)
    h = layout(v["idx"], worst)
    rx, _, rw, meta = ep.dispatch(h, v["y"], v["w"], zero_padding=True)
    rows = ep.expert_rows(h)
    R = h.total_rows
    new = lambda *shape: torch.zeros(shape, dtype=BF16, device=DEV)
    v["pre"], v["act"], v["out"] = new(R, 2 * F), new(R, F), new(R, H)
    ep.matmul(rx, gate_up, rows=rows, gated=True, pre=v["pre"], out=v["act"])
    ep.matmul(v["act"], down, rows=rows, out=v["out"])
    v["combined"] = ep.combine(h, v["out"], v["w"], bias=v["total"])
    # back: the gradient of combine is a dispatch, of dispatch a combine
    g, _ = ep.dispatch_cached(h, grad_out, zero_padding=True)
    v["grad_w"] = torch.zeros(R, dtype=torch.float32, device=DEV)
    v["grad_w"] += (g.float() * v["out"].float()).sum(1)
    v["g"] = (g.float() * rw[:, None]).to(BF16)
    v["g_act"], v["g_rows"] = new(R, F), new(R, H)
    v["gw_down"], v["gw_up"] = torch.empty_like(down), torch.empty_like(gate_up, dtype=torch.float32)
    ep.matmul_backward(v["act"], down, v["g"], rows=rows, out=(v["g_act"], v["gw_down"]))
    ep.matmul_backward(rx, gate_up, v["g_act"], rows=rows, gated=True, pre=v["pre"], out=(v["g_rows"], v["gw_up"]))
    v["g_y"] = ep.combine(h, v["g_rows"])
    dst = h.tensor("dst_row").view(T, K).long()
    v["g_logits"] = ep.route_backward(rc, logits, v["idx"], v["grad_w"][dst.clamp(min=0)].contiguous())
    v["g_router"] = torch.empty(E, H, dtype=torch.float32, device=DEV)
    g_y2, _ = ep.matmul_backward(v["y"], router, v["g_logits"], out=(new(T, H), v["g_router"]))
    v["g_x"], v["g_wn"] = ep.rms_norm_backward(v["total"], wn, v["g_y"] + g_y2, grad_total=grad_out)
    return v, rows, rx, h


def test_training_layer_forward_and_backward():
    x, res, wn, router = randn(1, T, H), randn(2, T, H), 1 + 0.1 * randn(3, H, dtype=torch.float32), randn(4, E, H)
    gate_up, down = randn(5, E, 2 * F, H, size=H ** -0.5), randn(6, E, H, F, size=F ** -0.5)
    v, rows, rx, h = training_step(x, res, wn, router, gate_up, down, randn(7, T, H))
    for e, (s, n) in enumerate(spans(*(t.tolist() for t in rows))):
        at = slice(s, s + n)
        if n == 0:
            assert not v["gw_down"][e].any() and not v["gw_up"][e].any()
            continue
        ref, tol, y, tol_y = expected(f64(rx[at]), f64(gate_up[e]), True, BF16)
        assert_close(v["act"][at], ref, tol, "act")
        assert_close(v["pre"][at], y, tol_y, "pre")
        ref, tol, _, _ = expected(f64(v["act"][at]), f64(down[e]), False, BF16)
        assert_close(v["out"][at], ref, tol, "out")
        d, off = product_gradient(f64(v["g"][at]), None, BF16)
        close_product(v["g_act"][at], d, f64(down[e]).T.copy(), off, BF16, "g_act")
        close_product(v["gw_down"][e], d.T.copy(), f64(v["act"][at]).T.copy(), off.T.copy(), BF16, "gw_down")
        d, off = product_gradient(f64(v["g_act"][at]), f64(v["pre"][at]), BF16)
        close_product(v["g_rows"][at], d, f64(gate_up[e]).T.copy(), off, BF16, "g_rows")
        close_product(v["gw_up"][e], d.T.copy(), f64(rx[at]).T.copy(), off.T.copy(), BF16, "gw_up")
    for name in ("g_x", "g_wn", "g_router", "combined"):
        assert v[name].isfinite().all()
    h.free()


def test_captured_layers_replay_as_eager():
    """Fixed windows: nothing is read back, so a training step and an E4M3 layer are captured whole."""
    x, res, wn, router = randn(1, T, H), randn(2, T, H), 1 + 0.1 * randn(3, H, dtype=torch.float32), randn(4, E, H)
    gate_up, down, g = randn(5, E, 2 * F, H, size=H ** -0.5), randn(6, E, H, F, size=F ** -0.5), randn(7, T, H)
    up8, down8 = weight_pair(5, 2 * F, H, True), weight_pair(6, H, F, False)
    rc, worst = ep.RouteConfig(E=E, K=K), T * K + E * 16
    h = layout(torch.zeros(T, K, dtype=torch.int64, device=DEV) + torch.arange(K, device=DEV), worst)
    new = lambda *shape: torch.zeros(shape, dtype=BF16, device=DEV)

    def step():
        y, q, total = ep.rms_norm(x, wn, residual=res, fp8=True)
        idx, w = ep.route(rc, ep.matmul(y, router))
        ep.relayout(h, idx)
        rx, rs, _, _ = ep.dispatch(h, q, w, zero_padding=True)
        rows, R = ep.expert_rows(h), h.total_rows
        act = ep.matmul_fp8((rx, rs), up8, rows=rows, gated=True, out=new(R, F))
        out8 = ep.combine(h, ep.matmul_fp8(ep.quantize_fp8(act), down8, rows=rows, out=new(R, H)), w, bias=total)
        rb, _, rw, _ = ep.dispatch(h, y, w, zero_padding=True)
        pre, a16 = new(R, 2 * F), new(R, F)
        ep.matmul(rb, gate_up, rows=rows, gated=True, pre=pre, out=a16)
        out16 = ep.combine(h, ep.matmul(a16, down, rows=rows, out=new(R, H)), w, bias=total)
        gr, _ = ep.dispatch_cached(h, g, zero_padding=True)
        ga, gd = ep.matmul_backward(a16, down, gr, rows=rows, out=(new(R, F), torch.empty_like(down)))
        gx, gu = ep.matmul_backward(rb, gate_up, ga, rows=rows, gated=True, pre=pre, out=(new(R, H), torch.empty_like(gate_up)))
        return [out8, out16, gd, gu, *ep.rms_norm_backward(total, wn, ep.combine(h, gx), grad_total=g)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(randn(20 + k, T, H))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    h.free()


def test_refusals_before_any_launch():
    x, w = randn(1, 8, 64), randn(2, 32, 64)
    for bad in (lambda: ep.rms_norm(x, w[0].cpu()), lambda: ep.rms_norm(x.cpu(), w[0]), lambda: ep.rms_norm(x, w[0, :63]),
                lambda: ep.rms_norm(x, w[0], residual=x[:7]), lambda: ep.rms_norm(x, w[0], keep=False),
                lambda: ep.rms_norm(x.t(), randn(1, 8)), lambda: ep.rms_norm_backward(x, w[0], x[:, :63]),
                lambda: ep.matmul(x, w[:, :32].contiguous()), lambda: ep.matmul(x[:, ::2], w[:, ::2]),
                lambda: ep.matmul(x, randn(2, 33, 64), gated=True), lambda: ep.matmul(x, w, pre=x),
                lambda: ep.matmul(x, w[None], rows=as_rows([0, 1], [1, 1])),
                lambda: ep.matmul_backward(x, w, randn(3, 8, 16), gated=True),
                lambda: ep.matmul_backward(x, w, randn(3, 8, 31)),
                lambda: ep.matmul_backward(x, w, randn(3, 8, 32), out=(None, None)),
                lambda: ep.matmul_backward(x, w, randn(3, 8, 32), out=(None, torch.empty(33, 64, device=DEV))),
                lambda: ep.quantize_fp8(x, out=(torch.empty(8, 64, dtype=torch.uint8, device=DEV),
                                                torch.empty(1, 8, device=DEV)))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ep.rms_norm(x, w[0].half()), lambda: ep.rms_norm(x, w[0], residual=x.float()),
                lambda: ep.rms_norm(x.double(), w[0].double()), lambda: ep.matmul(x.float(), w.float()),
                lambda: ep.matmul(x, w.half()), lambda: ep.matmul_fp8((x, x), (w, w)), lambda: ep.matmul_fp8(x, w),
                lambda: ep.matmul_backward(x, w, randn(3, 8, 32), out=(None, w.half())),
                lambda: ep.matmul_backward(x, w, randn(3, 8, 32), out=(None, 1.0)),
                lambda: ep.rms_norm(x, w[0], out=[x, None, None]), lambda: ep.quantize_fp8([1.0])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ep.rms_norm(x, w[0], eps=0.0), lambda: ep.matmul_backward(x, randn(2, 12, 64), randn(3, 8, 12)),
                lambda: ep.matmul(randn(1, 8, 60), randn(2, 32, 60))):
        with pytest.raises(ep.EpError):
            bad()
    assert ep.rms_norm(x[:0], w[0], fp8=True)[1][0].shape == (0, 64)
    assert ep.quantize_fp8(x[:0])[1].shape == (0, 1) and ep.matmul(x[:0], w).shape == (0, 32)
