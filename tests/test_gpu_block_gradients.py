"""Gradients of the calls that leave an operand out."""
import pytest
import torch

import block_refs as R
from block_refs import check
from gpu_helpers import log
from test_gpu_block import DEV, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pdtype", [None, torch.float32])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,d", [(90, 72), (5, 9000), (0, 16)])
def test_layer_norm_with_a_bias_alone(gpu_lib, rows, d, dtype, pdtype):
    fk = gpu_lib
    pdtype = pdtype or dtype
    log(f"bias alone {rows} x {d} {dtype} {pdtype}")
    X, dY, b = rand(rows, d, seed=1, dtype=dtype), rand(rows, d, seed=2, dtype=dtype), rand(d, seed=3, dtype=pdtype)
    Y, mean, rstd = fk.fk_layer_norm(X, bias=b)
    y, _, _, e_y, *_ = R.layer_norm(X, None, b, 1e-5)
    check("Y", Y, y, e_y, dtype)
    dX, dw, db = fk.fk_layer_norm_backward(dY, X, mean, rstd, bias_dtype=pdtype)
    want, _, sums, e_dx, _, e_db = R.layer_norm_grad(dY, X, None, 1e-5)
    assert dw is None and db.dtype == pdtype
    check("dX", dX, want, e_dx, dtype)
    check("dbias", db, sums, e_db, pdtype)
    assert fk.fk_layer_norm_backward(dY, X, mean, rstd, with_bias=False, bias_dtype=pdtype)[2] is None


def test_layer_norm_bias_type_refusals(gpu_lib):
    fk = gpu_lib
    X = rand(4, 32, seed=1, dtype=torch.bfloat16)
    w = torch.ones(32, device=DEV)
    _, mean, rstd = fk.fk_layer_norm(X, w)
    with pytest.raises(ValueError):
        fk.fk_layer_norm_backward(X, X, mean, rstd, bias_dtype=torch.float16)
    with pytest.raises(ValueError):
        fk.fk_layer_norm_backward(X, X, mean, rstd, w, bias_dtype=torch.bfloat16)
    assert fk.fk_layer_norm_backward(X, X, mean, rstd, w, bias_dtype=torch.float32)[2].dtype == torch.float32


@pytest.mark.parametrize("rows,k,d", [(40, 3, 96), (7, 9, 2052), (3, 2, 9001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine_without_gates(gpu_lib, rows, k, d, dtype):
    """The gradient of a plain sum: every slot gets its row's."""
    fk = gpu_lib
    log(f"combine without gates {rows} x {k} x {d} {dtype}")
    dOut, Y = rand(rows, d, seed=1, dtype=dtype), rand(rows * k, d, seed=2, dtype=dtype)
    dY, dgates = fk.fk_combine_backward(dOut, Y, None)
    assert dgates is None and torch.equal(dY, dOut.repeat_interleave(k, 0))
    with pytest.raises(ValueError):
        fk.fk_combine_backward(dOut, Y[1:], None)
