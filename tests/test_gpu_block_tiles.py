"""Products of enough rows and columns for the tiles of 256, with everything in
their epilogue and with rows by slots, against 64 bits."""
import pytest
import torch

import block_refs as R
from block_refs import check
from gpu_helpers import log
from test_gpu_block import DEV, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,name", [(2500, 4104, 200, "gelu"), (2304, 4352, 72, "silu")])
def test_large_tiles_with_residual_and_pre(gpu_lib, M, N, K, name, dtype):
    """170 and 153 tiles of 256 (the latter are of 128 then): whole ones and
    those that end within the matrix; the residual by itself and in place."""
    fk = gpu_lib
    log(f"linear {M} x {N} x {K} {dtype} {name}")
    X, Wt = rand(M, K, seed=1, dtype=dtype), rand(N, K, seed=2, scale=K ** -0.5, dtype=dtype)
    b, res = rand(N, seed=3, dtype=dtype), rand(M, N, seed=4, dtype=dtype)
    y, z, e_y, e_z = R.linear(X, Wt, b, name, res)
    Y, pre = fk.fk_linear(X, Wt, b, act=name, residual=res, with_pre=True)
    check("Y", Y, y, e_y, dtype)
    check("pre", pre, z, e_z, dtype)
    again, _ = fk.fk_linear(X, Wt, b, act=name, residual=res)
    assert torch.equal(again, Y)
    wide, _ = fk.fk_linear(X, Wt, b, act=name, residual=res, out_dtype=torch.float32)
    check("fp32 Y", wide, y, e_y, torch.float32)
    got, _ = fk.fk_linear(X, Wt, b, act=name, residual=res, Y=res)
    assert got is res and torch.equal(got, Y)


def _ids(T, share, E, seed):
    """Uneven loads: group 2 empty, group 5 of 100 slots, some slots unrouted."""
    g = torch.Generator().manual_seed(seed)
    ids = (E * torch.rand(T * share, generator=g) ** 1.5).long().clamp_max(E - 1)
    ids[ids == 2] = 3
    ids[ids == 5] = 6
    ids[torch.randperm(T * share, generator=g)[:100]] = 5
    ids[torch.randperm(T * share, generator=g)[:77]] = E
    return ids.to(torch.int32).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("share,name,N,K", [(2, "silu", 1280, 1280), (1, "none", 1288, 1304)])
def test_large_tiles_by_slots(gpu_lib, share, name, N, K, dtype):
    """Eight groups of a thousand slots each on average: forward with X read by
    slots / share, dX from dZ in order (silu) and from dY by slots (none), dW
    with sums from none to thousands of positions."""
    fk = gpu_lib
    E, M = 8, 8008
    T = M // share
    log(f"grouped {T} x {share} over {E}, {N} x {K} {dtype} {name}")
    ids = _ids(T, share, E, share)
    slots, offsets = fk.fk_sort_inverse(ids, E + 1)
    where = {"slots": slots, "offsets": offsets, "share": share}
    X, Wt = rand(T, K, seed=1, dtype=dtype), rand(E, N, K, seed=2, scale=K ** -0.5, dtype=dtype)
    b, res = rand(E, N, seed=3, dtype=dtype), rand(M, N, seed=4, dtype=dtype)
    y, z, e_y, e_z = R.linear(X, Wt, b, name, res, **where)
    Y, pre = fk.fk_linear(X, Wt, b, act=name, residual=res, with_pre=True, **where)
    check("Y", Y, y, e_y, dtype)
    check("pre", pre, z, e_z, dtype)
    assert not Y[ids == E].any()
    dY = rand(M, N, seed=5, dtype=dtype)
    kept = None if name == "none" else pre
    dx, dw, db, e_dx, e_dw, e_db = R.linear_grad(dY, X, Wt, name, kept, **where)
    dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, act=name, pre=kept, **where)
    check("dX", dX, dx, e_dx, dtype)
    check("dW", dW, dw, e_dw, dtype)
    check("dbias", dB, db, e_db, dtype)
    assert not dW[2].any() and not dX[ids == E].any()
