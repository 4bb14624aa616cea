"""Each width of the norm's kernels and of its gradient's at the rows that choose it, teams that take many rows one
after the other among them.  Plain implementation and tolerances are those of test_norm.py."""

import pytest
import torch

from test_norm import DTYPES, check_backward, check_norm, randn, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# rows for more and for less than all CUs, widths around the pieces of 16 bytes that change the lanes
@pytest.mark.parametrize("N", [7, 256, 257, 1023, 1025])
@pytest.mark.parametrize("pieces", [15, 16, 17, 33, 64, 65, 128, 129, 257, 513, 1023, 1024, 1025])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_norm_at_every_width(N, pieces, dtype):
    t = DTYPES[dtype]
    V = 16 // torch.empty(0, dtype=t).element_size()
    H = pieces * V - (N % 2)  # odd rows' last piece is not whole
    say("width", N, H, dtype)
    x, r = 3 * randn(N + H, N, H, dtype=t), randn(N + H + 1, N, H, dtype=t)
    x[N // 2] = 0
    check_norm(x, 1 + 0.1 * randn(H, H), r, fp8=True)
    check_norm(x, (1 + 0.1 * randn(H, H)).to(t))


# few workgroups take many rows each: with the next row ahead and without, and many rows in all
@pytest.mark.parametrize("N,H", [(70000, 8), (40000, 136), (9000, 513), (2500, 1000), (3001, 2048), (3000, 4100), (1030, 7168),
                                 (900, 8192), (800, 8200), (777, 16384), (520, 20001), (600, 32768)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_backward_of_many_rows_a_team(N, H, dtype):
    t = DTYPES[dtype]
    say("many rows", N, H, dtype)
    x, g, p = 3 * randn(N + H, N, H, dtype=t), randn(N + H + 1, N, H, dtype=t), randn(N, N, H, dtype=t)
    x[N // 3] = 0
    x[N // 2] *= 2.0 ** -10
    check_backward(x, 1 + 0.1 * randn(1, H), g, through=p)
    check_backward(x, (1 + 0.1 * randn(1, H)).to(t), g)


@pytest.mark.parametrize("H", [100, 1024, 2048, 4096, 8192, 16384])
def test_backward_of_rows_that_leave_fp32_among_others(H):
    """A team's row of squares beyond fp32 between ordinary ones, on teams of one and of several waves."""
    N = 6 * 1280 if H <= 1024 else 1800
    x, g, w = randn(1, N, H), randn(2, N, H), randn(3, H)
    for k, s in ((5, 1e25), (256 + 5, 1e30), (512 + 5, 1e-30), (600, 1e25), (N - 1, 1e25)):
        x[k] *= s
    for eps in (1e-6, 1e-30):
        say("leave", H, eps)
        check_backward(x, w, g, eps=eps)
