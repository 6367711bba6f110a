"""Operands that are slices of one buffer, or that start off 16 bytes."""
import pytest
import torch

import block_refs as R
from block_refs import check
from gpu_helpers import log
from test_gpu_block import rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 57])
def test_outputs_beside_inputs(gpu_lib, d, dtype):
    """Input, output and a third slice, columns of one buffer each."""
    fk = gpu_lib
    log(f"slices of {d} {dtype}")
    buf = rand(70, 3 * d, seed=d, dtype=dtype)
    a, b, c = (buf[:, i * d:(i + 1) * d] for i in range(3))
    x, other = a.clone(), c.clone()
    want, mean, rstd = fk.fk_layer_norm(x)
    assert fk.fk_layer_norm(a, Y=b)[0] is b
    assert torch.equal(b, want) and torch.equal(a, x) and torch.equal(c, other)
    dx, _, _ = fk.fk_layer_norm_backward(other, x, mean, rstd)
    assert torch.equal(fk.fk_layer_norm_backward(c, a, mean, rstd, dX=b)[0], dx)
    assert torch.equal(b, dx) and torch.equal(a, x) and torch.equal(c, other)
    Y = rand(140, d, seed=3, dtype=dtype)
    assert torch.equal(fk.fk_combine(Y, 2, residual=a, out=b), fk.fk_combine(Y, 2, residual=x))
    assert torch.equal(a, x) and torch.equal(c, other)
