"""Products at the sizes where their rules turn: 32 columns a workgroup for a
few rows, sums split in other than powers of two, split sums over more than one
round of tiles (fp32), the fewest large tiles.  Against float64 on the GPU, each
output within the rounding of a sum of that length and of its type."""
import pytest
import torch

import block_refs as R
from test_gpu_block import check, log, rand

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dense(fk, M, N, K, dtype):
    log(f"linear {M} x {N} x {K} {dtype}")
    X, Wt = rand(M, K, seed=1, dtype=dtype), rand(N, K, seed=2, scale=K ** -0.5, dtype=dtype)
    b, res, dY = rand(N, seed=3, dtype=dtype), rand(M, N, seed=4, dtype=dtype), rand(M, N, seed=5, dtype=dtype)
    x, w, dy = X.double(), Wt.double(), dY.double()
    z = x @ w.t() + b.double()
    Y, _ = fk.fk_linear(X, Wt, b, act="relu", residual=res)
    e = (K + 24) * R.W * (x.abs() @ w.abs().t() + b.double().abs() + res.double().abs())
    check("Y", Y, (z.relu() + res.double()).cpu(), e.cpu(), dtype)
    dX, dW, dB = fk.fk_linear_backward(dY, X, Wt)
    check("dX", dX, (dy @ w).cpu(), ((N + 24) * R.W * (dy.abs() @ w.abs())).cpu(), dtype)
    check("dW", dW, (dy.t() @ x).cpu(), ((M + 24) * R.W * (dy.abs().t() @ x.abs())).cpu(), dtype)
    check("dbias", dB, dy.sum(0).cpu(), ((M + 24) * R.W * dy.abs().sum(0)).cpu(), dtype)


@pytest.mark.parametrize("M,N,K", [(1, 65541, 40), (16, 65536, 72), (300, 500, 3000), (2056, 4700, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense(gpu_lib, M, N, K, dtype):
    _dense(gpu_lib, M, N, K, dtype)


def test_split_sums_of_several_rounds(gpu_lib):
    _dense(gpu_lib, 2000, 2600, 4100, torch.float32)


@pytest.mark.parametrize("E,N,rows", [(520, 130, 2000), (64, 1030, 500)])
def test_few_rows_of_many_groups(gpu_lib, E, N, rows):
    """Groups from empty to more than the 16 rows that are taken as few."""
    fk = gpu_lib
    K, dtype = 48, torch.bfloat16
    log(f"groups {E} x {N} x {K}, {rows} rows")
    g = torch.Generator().manual_seed(E)
    ids = (E * torch.rand(rows, generator=g) ** 3).long().to(torch.int32).to(DEV)
    loads = torch.bincount(ids.long(), minlength=E)
    assert int(loads.min()) == 0 and int(loads.max()) > 16
    slots, offsets = fk.fk_sort_inverse(ids, E + 1)
    X, Wt = rand(rows, K, seed=1, dtype=dtype), rand(E, N, K, seed=2, scale=K ** -0.5, dtype=dtype)
    Y, _ = fk.fk_linear(X, Wt, slots=slots, offsets=offsets)
    x, w = X.double(), Wt.double()
    y, e = torch.empty((2, rows, N), dtype=torch.float64, device=DEV)
    for i in range(E):
        mine = ids == i
        y[mine] = x[mine] @ w[i].t()
        e[mine] = (K + 24) * R.W * (x[mine].abs() @ w[i].abs().t())
    check("Y", Y, y.cpu(), e.cpu(), dtype)
