"""Products of one column and more rows than one dimension of a launch has tiles
for (2^24 workgroups of 256 threads)."""
import pytest
import torch

from gpu_helpers import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_bias_gradient_of_two_to_the_thirty_rows(gpu_lib):
    """A sum of ones: the tiles' and the threads' sums are multiples of 64 up to
    2^30, exact in fp32, and so is the result."""
    fk = gpu_lib
    M = (1 << 30) + 128
    log(f"db of {M} rows")
    dY = torch.ones((M, 1), dtype=torch.bfloat16, device=DEV)
    W = torch.ones((1, 1), dtype=torch.bfloat16, device=DEV)
    db = fk.fk_linear_backward(dY, dY.clone(), W, with_dx=False, with_dw=False, bias_dtype=torch.float32)[2]
    assert float(db) == M


def test_all_the_rows_there_may_be(gpu_lib):
    """fp32, whose tiles are of 128 rows: each row's product is its own."""
    fk = gpu_lib
    M = (1 << 31) - 1
    log(f"forward of {M} rows")
    X = torch.empty((M, 1), device=DEV)
    for i in range(0, M, 1 << 28):
        n = min(1 << 28, M - i)
        X[i:i + n, 0] = (torch.arange(n, device=DEV) % 8191).float() + float(i >> 28)
    W, b = torch.full((1, 1), 3.0, device=DEV), torch.full((1,), 0.5, device=DEV)
    Y, _ = fk.fk_linear(X, W, b)
    for i in range(0, M, 1 << 28):
        assert torch.equal(Y[i:i + (1 << 28)], X[i:i + (1 << 28)] * 3 + 0.5), i
    fk._ws_cache.clear()
