"""A recorded expert block beside eager work of the same stream that needs more
scratch than the recorded calls."""
import pytest
import torch

from gpu_helpers import log
from test_gpu_block import _block, _block_params, rand

pytestmark = pytest.mark.gpu


def test_graph_keeps_its_scratch_while_the_stream_grows(gpu_lib):
    fk = gpu_lib
    p = _block_params(4, 136, 200, torch.bfloat16)
    small, large = (rand(n, 136, seed=n, dtype=torch.bfloat16) for n in (90, 5000))
    _block(fk, small, p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    log("recording")
    with torch.cuda.graph(graph, stream=s):
        got = _block(fk, small, p)
    # more scratch on the stream of the recording, before and between replays
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want_large = [t.clone() for t in _block(fk, large, p)]
    torch.cuda.synchronize()
    filled = [torch.full((n,), 7, dtype=torch.uint8, device="cuda:0") for n in (1 << 10, 1 << 16, 1 << 20, 1 << 24) for _ in range(8)]
    for seed in (3, 4, 3):
        log(f"replay {seed}")
        small.copy_(rand(90, 136, seed=seed, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in filled)
        for u, v in zip(got, _block(fk, small.clone(), p)):
            assert torch.equal(u, v)
        with torch.cuda.stream(s):
            for u, v in zip(_block(fk, large, p), want_large):
                assert torch.equal(u, v)
        torch.cuda.synchronize()
