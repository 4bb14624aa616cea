"""Host-side queries of the kernels that the E4M3 and 16-bit products and the gradients take.  CPU only."""

import ctypes
import os

import pytest
import torch

import combine_topk_idx_expert_amd as ep

S = ep.Status


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ep.lib_path()):
        import combine_topk_idx_expert_amd.build as b

        b.build()
    return ep.lib()


def test_product_kernels(L):
    assert ep.debug_product_kernels(0, 0, 64) == ()
    assert ep.debug_product_kernels(64, 0, 49152) == ("split",)
    # dense: the height that costs fewer rounds, whatever int8 takes
    assert ep.debug_product_kernels(22240, 0, 326, gated=True) == ("tiles256",)
    assert ep.debug_matmul_kernels(22240, 0, 326, gated=True) == ("tiles128",)
    assert ep.debug_product_kernels(65, 0, 49152) == ("tiles128",) and ep.debug_matmul_kernels(65, 0, 49152) == ("tiles256",)
    # groups: as int8
    for M, G, N in ((576, 32, 4096), (6000, 64, 4096), (20000, 64, 4096), (9000, 4, 512)):
        assert ep.debug_product_kernels(M, G, N) == ep.debug_matmul_kernels(M, G, N)
    # fp32 results of E4M3 rows take no tiles of 256 rows
    for M, G, N in ((6000, 64, 4096), (20000, 64, 4096), (8192, 0, 8192)):
        assert "tiles256" in ep.debug_product_kernels(M, G, N)
        assert ep.debug_product_kernels(M, G, N, dtype=torch.float32) == tuple(
            n.replace("256", "128") for n in ep.debug_product_kernels(M, G, N))
    bits = ctypes.c_uint32()
    assert L.ep_debug_product_kernels(1, 0, 64, 0, 1, None) == S.ERR_NULL
    assert L.ep_debug_product_kernels(1, 0, 64, 0, 3, ctypes.byref(bits)) == S.ERR_SHAPE
    assert L.ep_debug_product_kernels(1, 0, 63, 1, 1, ctypes.byref(bits)) == S.ERR_SHAPE
    assert L.ep_debug_product_kernels(1 << 31, 0, 64, 0, 1, ctypes.byref(bits)) == S.ERR_OVERFLOW


def test_backward_plan_is_what_the_workspace_holds(L):
    plan, size = (ctypes.c_int32 * 4)(), ctypes.c_int64()
    for M, G, K, N, gated in ((1, 0, 4096, 4096, True), (32768, 0, 512, 512, False), (18090, 8, 960, 288, True),
                              (153, 3, 256, 4096, False), (65536, 32, 4096, 4096, True), (300, 0, 3584, 4096, False)):
        (rt, rs), (wt, ws) = ep.debug_backward_plan(M, G, K, N, gated)
        assert {rt, wt} <= {128, 256} and (rs == 1 or rt == 128) and (ws == 1 or wt == 128)
        assert L.ep_matmul_backward_workspace(M, G, K, N, int(gated), ctypes.byref(size)) == S.OK
        slices = max(rs * M * K * 4 if rs > 1 else 0, ws * max(G, 1) * N * K * 4 if ws > 1 else 0)
        assert size.value == slices + ((M * N * 2 + 255) // 256 * 256 if gated else 0)
    assert L.ep_debug_backward_plan(1, 0, 64, 64, 0, None) == S.ERR_NULL
    assert L.ep_debug_backward_plan(1, 0, 64, 36, 0, plan) == S.ERR_SHAPE
    assert L.ep_debug_backward_plan(1 << 31, 0, 64, 64, 0, plan) == S.ERR_OVERFLOW
