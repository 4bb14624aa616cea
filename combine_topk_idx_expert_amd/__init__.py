"""MoE dispatch / combine on one MI355X: Python binding of libep_mi355x.so.

The binding only marshals arguments: it allocates output tensors with torch
(device memory is torch's plumbing), passes raw device pointers and torch's
current stream to the C ABI of ``include/ep_mi355x.h``, and turns status codes
into exceptions.  Every step of the path runs in the library's HIP kernels;
there is no fallback: if the library is missing, importing works but every
call raises.

    h = get_layout(Config(P, S, H, K, E, A), topk_idx)       # plan (syncs once)
    recv_x, recv_scales, recv_w, meta = dispatch(h, x, topk_weights, fp8=False,
                                                 zero_padding=True)
    y = experts(recv_x, ...)                                  # caller's work
    out = combine(h, y, topk_weights)
    h.free()

Around it: the router (route, route_backward), the norm (rms_norm, rms_norm_backward), quantising
(quantize_int8, quantize_fp8) and the experts' products (matmul_int8, matmul_fp8, matmul,
matmul_backward).
"""

from __future__ import annotations

from ._native import (  # noqa: F401
    EP_ABI_VERSION,
    Config,
    EpError,
    EventOverlap,
    Handle,
    LibraryMissing,
    RouteConfig,
    STATUS_ROUTING,
    STATUS_TRUNCATED,
    Status,
    TENSORS,
    buffer_size_hint,
    combine,
    comm_stream,
    debug_backward_plan,
    debug_copy,
    debug_e4m3_encode,
    debug_matmul_kernels,
    debug_product_kernels,
    debug_split_shape,
    dispatch,
    dispatch_cached,
    expert_rows,
    get_layout,
    lib,
    lib_path,
    matmul,
    matmul_backward,
    matmul_fp8,
    matmul_int8,
    quantize_fp8,
    quantize_int8,
    rms_norm,
    rms_norm_backward,
    relayout,
    route,
    route_backward,
)
