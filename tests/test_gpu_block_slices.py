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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(5, 33, 67), (90, 131, 257)])
def test_rows_cut_from_odd_matrices(gpu_lib, M, N, K, dtype):
    """X[1:], W[1:], dY[1:] and pre[1:] with odd widths: none starts on 16 bytes."""
    fk = gpu_lib
    log(f"cut rows {M} x {N} x {K} {dtype}")
    X, Wt = rand(M + 1, K, seed=1, dtype=dtype)[1:], rand(N + 1, K, seed=2, scale=K ** -0.5, dtype=dtype)[1:]
    b, res = rand(N, seed=3, dtype=dtype), rand(M + 1, N, seed=4, dtype=dtype)[1:]
    dY, pre = rand(M + 1, N, seed=5, dtype=dtype)[1:], rand(M + 1, N, seed=6, dtype=dtype)[1:]
    assert all(t.data_ptr() % 16 for t in (X, Wt, res, dY, pre))
    y, _, e_y, _ = R.linear(X, Wt, b, "silu", res)
    check("Y", fk.fk_linear(X, Wt, b, act="silu", residual=res)[0], y, e_y, dtype)
    for name in ("silu", "none"):
        kept = pre if name == "silu" else None
        dx, dw, db, e_dx, e_dw, e_db = R.linear_grad(dY, X, Wt, name, kept)
        dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, act=name, pre=kept)
        check("dX", dX, dx, e_dx, dtype)
        check("dW", dW, dw, e_dw, dtype)
        check("dbias", dB, db, e_db, dtype)


def test_pre_off_16_bytes(gpu_lib):
    """Whole chunks in pre's rows that start on no chunk."""
    fk = gpu_lib
    M, N, K = 130, 512, 64
    X, Wt, dY = rand(M, K, seed=1), rand(N, K, seed=2, scale=0.1), rand(M, N, seed=3)
    pre = rand(M * N + 1, seed=4)[1:].view(M, N)
    for got, want in zip(fk.fk_linear_backward(dY, X, Wt, act="gelu", pre=pre),
                         fk.fk_linear_backward(dY, X, Wt, act="gelu", pre=pre.clone())):
        assert torch.equal(got, want)


def test_rows_in_order_past_2_gib(gpu_lib):
    """Groups of rows that lie in order, X and dY past 2 GiB each: read as they
    lie, with scratch that holds neither.  Samples against float64."""
    fk = gpu_lib
    E, M, N, K, dtype = 3, 1_050_007, 1032, 1032, torch.bfloat16
    g = torch.Generator(device="cuda:0").manual_seed(1)
    X, dY = (torch.empty((M, K), dtype=dtype, device="cuda:0").normal_(generator=g) for _ in range(2))
    assert X.numel() * 2 > 1 << 31
    Wt = rand(E, N, K, seed=2, scale=K ** -0.5, dtype=dtype)
    cuts = [0, 300_001, 300_001, M - 11]  # the second group empty, eleven rows past the last
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda:0")
    scratch = torch.empty(1 << 30, dtype=torch.uint8, device="cuda:0")
    log("forward")
    Y, _ = fk.fk_linear(X, Wt, offsets=offsets, workspace=scratch)
    log("backward")
    dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, offsets=offsets, workspace=scratch)
    assert not dW[1].any() and not dB[1].any()
    for e in (0, 2):
        lo, hi = cuts[e], cuts[e + 1]
        at = torch.cat((torch.arange(lo, hi, 40009, device="cuda:0"), torch.arange(hi - 3, hi, device="cuda:0")))
        x, d, w = X[at].double(), dY[at].double(), Wt[e].double()
        check(f"Y of {e}", Y[at], (x @ w.t()).cpu(), ((K + 24) * R.W * (x.abs() @ w.abs().t())).cpu(), dtype)
        check(f"dX of {e}", dX[at], (d @ w).cpu(), ((N + 24) * R.W * (d.abs() @ w.abs())).cpu(), dtype)
        want, mag = (torch.zeros((8, K), dtype=R.D, device="cuda:0") for _ in range(2))
        for i in range(lo, hi, 100_000):
            d, x = dY[i:min(i + 100_000, hi), :8].double(), X[i:min(i + 100_000, hi)].double()
            want += d.t() @ x
            mag += d.abs().t() @ x.abs()
        check(f"dW of {e}", dW[e, :8], want.cpu(), ((hi - lo + 24) * R.W * mag).cpu(), dtype)
    assert not Y[M - 11:].any() and not dX[M - 11:].any()
