"""The expert block as the example trains and uses it."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py")
    spec = importlib.util.spec_from_file_location("expert_block_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_error(gpu_lib):
    ex = _example()
    block, x, history = ex.train(steps=40, rows=4096, dim=128, experts=8, log=lambda m: print(m, flush=True))
    assert torch.isfinite(history).all()
    assert float(history[-5:].mean()) < 0.5 * float(history[:5].mean())
    with torch.no_grad():
        whole, losses, counts = block(x)
        assert int(counts.sum()) == 2 * x.shape[0] and torch.isfinite(losses).all()
        # a row by itself: the same products in another order of summation, so
        # equal to a few roundings of bf16 on the way (three products and their
        # sum, each within 2^-8 of values below max |out|), unless the row's
        # second choice was nearly tied
        some = torch.cat([block(x[i:i + 1])[0] for i in range(8)])
        off = (some - whole[:8]).abs().max(1)[0] <= 4 * 2.0 ** -8 * whole.abs().max()
        assert int(off.sum()) >= 7
