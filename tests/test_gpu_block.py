"""The expert-block operators on the GPU against their 64-bit definitions
(block_refs.py, which also derives the bounds): sizes from one row and one
column to ragged ones past every tile, each type, strided rows, masks that
leave a row empty, empty and uneven groups, unrouted slots, gradients against
the formulas and against differences, repeatability, other streams, graphs."""
import math

import pytest
import torch

import block_refs as R
from block_refs import check
from gpu_helpers import log

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
DEV = "cuda:0"


def rand(*shape, seed, scale=1.0, dtype=torch.float32, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(DEV)


def strided(t, extra):
    """The same matrix with rows `extra` elements further apart, NaN between."""
    out = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    out[:, :t.shape[1]] = t
    return out[:, :t.shape[1]]


# ---- layer norm -----------------------------------------------------------------

NORM_SIZES = [(1, 1), (3, 7), (5, 64), (1, 512), (70, 513), (33, 768), (129, 1000), (2, 2048), (17, 2056), (9, 4096),
              (6, 4100), (700, 72), (3000, 8), (5, 8192), (4, 8193), (3, 20000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", NORM_SIZES)
def test_layer_norm(gpu_lib, rows, d, dtype):
    fk = gpu_lib
    log(f"layer norm {rows} x {d} {dtype}")
    X = rand(rows, d, seed=rows + d, scale=2.0, shift=1.5, dtype=dtype)
    dY = rand(rows, d, seed=rows + d + 1, dtype=dtype)
    w = rand(d, seed=d, scale=0.3, shift=1.0, dtype=dtype)
    b = rand(d, seed=d + 9, dtype=dtype)
    y, mu, r, e_y, e_mu, _, rel_r = R.layer_norm(X, w, b, 1e-5)
    Y, mean, rstd = fk.fk_layer_norm(X, w, b, eps=1e-5)
    check("Y", Y, y, e_y, dtype)
    check("mean", mean, mu, e_mu, torch.float32)
    check("rstd", rstd, r, rel_r * r, torch.float32)
    dx, dw, db, e_dx, e_dw, e_db = R.layer_norm_grad(dY, X, w, 1e-5)
    dX, dW, dB = fk.fk_layer_norm_backward(dY, X, mean, rstd, w)
    check("dX", dX, dx, e_dx, dtype)
    check("dweight", dW, dw, e_dw, dtype)
    check("dbias", dB, db, e_db, dtype)


@pytest.mark.parametrize("dtype,d,extra", [(torch.bfloat16, 768, 8), (torch.bfloat16, 96, 3), (torch.float32, 10, 6),
                                           (torch.float16, 9000, 24)])
def test_layer_norm_strides_and_fp32_parameters(gpu_lib, dtype, d, extra):
    fk = gpu_lib
    X = strided(rand(37, d, seed=3, shift=-4.0, dtype=dtype), extra)
    dY = strided(rand(37, d, seed=4, dtype=dtype), 2 * extra)
    w, b = rand(d, seed=5, shift=1.0), rand(d, seed=6)
    Y = strided(torch.zeros((37, d), dtype=dtype, device=DEV), extra)
    y, _, _, e_y, _, _, _ = R.layer_norm(X, w, b, 1e-3)
    got, mean, rstd = fk.fk_layer_norm(X, w, b, eps=1e-3, Y=Y)
    assert got is Y and torch.isnan(Y._base[:, d:]).all()
    check("Y", Y, y, e_y, dtype)
    dx, dw, db, e_dx, e_dw, e_db = R.layer_norm_grad(dY, X, w, 1e-3)
    dX, dW, dB = fk.fk_layer_norm_backward(dY, X, mean, rstd, w)
    assert dW.dtype == dB.dtype == torch.float32
    check("dX", dX, dx, e_dx, dtype)
    check("dweight", dW, dw, e_dw, torch.float32)
    check("dbias", dB, db, e_db, torch.float32)


def test_layer_norm_without_parameters_in_place_and_constant_rows(gpu_lib):
    fk = gpu_lib
    X = rand(50, 640, seed=1, dtype=torch.bfloat16)
    X[7] = 3.0   # no variance: rstd = eps^-1/2
    X[8] = 0.0
    y, _, r, e_y, _, _, rel = R.layer_norm(X, None, None, 1e-5)
    Y, mean, rstd = fk.fk_layer_norm(X)
    check("Y", Y, y, e_y, torch.bfloat16)
    check("rstd", rstd, r, rel * r, torch.float32)
    Z, _, _ = fk.fk_layer_norm(X, Y=X)
    assert Z is X and torch.equal(Z, Y)
    dY = rand(50, 640, seed=2, dtype=torch.bfloat16)
    dX, dw, db = fk.fk_layer_norm_backward(dY, Y, mean, rstd)
    assert dw is None and db is None
    dX2, _, _ = fk.fk_layer_norm_backward(dY, Y, mean, rstd, dX=dY)
    assert torch.equal(dX, dX2)


def test_layer_norm_nan_stays_in_its_row(gpu_lib):
    fk = gpu_lib
    X = rand(40, 256, seed=1)
    Y0, _, _ = fk.fk_layer_norm(X)
    X[11, 3] = float("nan")
    X[12, 5] = float("inf")
    Y1, _, _ = fk.fk_layer_norm(X)
    ok = torch.ones(40, dtype=torch.bool)
    ok[11:13] = False
    assert torch.equal(Y0[ok], Y1[ok]) and torch.isnan(Y1[11:13]).all(1).any()


def test_no_rows(gpu_lib):
    fk = gpu_lib
    X = torch.empty((0, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    Y, mean, rstd = fk.fk_layer_norm(X, w, w)
    assert Y.shape == (0, 64)
    dX, dw, db = fk.fk_layer_norm_backward(X, X, mean, rstd, w)
    assert dX.shape == (0, 64) and not dw.any() and not db.any()
    ids, gates, counts, losses, live = fk.fk_route(torch.empty((0, 5), device=DEV), 2)
    assert ids.shape == (0, 2) and not counts.any() and not losses.any() and int(live) == 0
    assert fk.fk_route_backward(torch.empty((0, 5), device=DEV), ids, counts, live).shape == (0, 5)
    Wt = rand(32, 64, seed=1)
    assert fk.fk_linear(X, Wt)[0].shape == (0, 32)
    dX, dW, db = fk.fk_linear_backward(torch.empty((0, 32), device=DEV), X, Wt)
    assert dX.shape == (0, 64) and not dW.any() and not db.any()
    assert fk.fk_combine(X, 2, torch.empty((0, 2), device=DEV)).shape == (0, 64)


# ---- router ------------------------------------------------------------------------

# probabilities: an exponential of a difference below 64 and the row's sum;
# losses: those and the sum over rows
P_REL = 120 * R.W

ROUTE_SIZES = [(1, 1, 1), (3, 2, 2), (5, 8, 2), (130, 7, 3), (64, 16, 16), (1000, 60, 6), (2049, 64, 8), (300, 128, 8),
               (77, 160, 6), (50, 256, 8), (20, 511, 4), (9, 1000, 33), (6, 1024, 64), (70000, 8, 1)]


def _route_case(T, E, k, dtype, masked, padded, seed):
    l = rand(T, E, seed=seed, scale=2.0, dtype=dtype)
    g = torch.Generator().manual_seed(seed + 1)
    valid = None
    if masked:
        m = torch.rand((T, E), generator=g) < 0.3
        m[0] = True                       # a row that the mask leaves empty
        m[T // 2, 1:] = True              # a row with one expert left
        l[m.to(DEV)] = -math.inf
    if padded:
        valid = (torch.rand(T, generator=g) > 0.25).to(DEV)
        l[~valid] = float("nan")          # what a padded row holds does not count
    return l, valid


@pytest.mark.parametrize("norm", ["chosen", "all"])
@pytest.mark.parametrize("masked,padded", [(False, False), (True, True)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", ROUTE_SIZES)
def test_route(gpu_lib, T, E, k, dtype, masked, padded, norm):
    fk = gpu_lib
    log(f"route {T} x {E} k={k} {dtype} masked={masked} {norm}")
    l, valid = _route_case(T, E, k, dtype, masked, padded, T + E + k)
    ids, gates, counts, losses, n, p, *_ = R.route(l, k, norm, valid)
    got = fk.fk_route(l, k, norm=norm, valid=valid)
    assert torch.equal(got[0].cpu(), ids)
    assert torch.equal(got[2].cpu(), counts)
    assert int(got[4]) == n
    check("gates", got[1], gates, P_REL * gates, torch.float32)
    check("losses", got[3], losses, (P_REL + (T + 60) * R.W) * losses, torch.float32)
    dg = rand(T, k, seed=T + 7)
    dl = torch.tensor([0.7, -0.3], device=DEV)
    want, mag = R.route_grad(l, k, norm, valid, dg, dl)
    d = fk.fk_route_backward(l, got[0], got[2], got[4], dg, dl, norm=norm, valid=valid)
    check("d_logits", d, want, 3 * P_REL * mag, dtype)
    d = fk.fk_route_backward(l, got[0], got[2], got[4], None, dl, norm=norm, valid=valid)
    check("d_logits of the losses", d, *_scaled(R.route_grad(l, k, norm, valid, None, dl)), dtype)
    d = fk.fk_route_backward(l, got[0], got[2], got[4], dg, None, norm=norm, valid=valid)
    check("d_logits of the gates", d, *_scaled(R.route_grad(l, k, norm, valid, dg, None)), dtype)


def _scaled(pair):
    return pair[0], 3 * P_REL * pair[1]


@pytest.mark.parametrize("E,k", [(8, 3), (64, 5), (200, 4), (1024, 9)])
def test_route_ties_go_to_the_lowest_index(gpu_lib, E, k):
    fk = gpu_lib
    g = torch.Generator().manual_seed(E)
    l = torch.randint(-2, 3, (500, E), generator=g).float().to(DEV)  # mostly ties
    l[3] = 0.0
    l[4] = torch.finfo(torch.float32).min  # the type's lowest value is a number like any other
    l[5, :] = -0.0
    l[5, 1] = 0.0
    ids, gates, counts, losses, n, *_ = R.route(l, k, "chosen")
    got = fk.fk_route(l, k)
    assert torch.equal(got[0].cpu(), ids) and torch.equal(got[2].cpu(), counts) and int(got[4]) == n == 500
    check("gates", got[1], gates, P_REL * gates, torch.float32)


def test_route_nan_and_inf(gpu_lib):
    """NaN is never chosen and reaches the losses; +inf is chosen first."""
    fk = gpu_lib
    l = rand(64, 32, seed=1)
    l[5, 2] = float("nan")
    l[6] = float("nan")
    l[7, 9] = float("inf")
    ids, gates, counts, losses, live = fk.fk_route(l, 4)
    want = R.route(l, 4, "chosen")
    assert torch.equal(ids.cpu(), want[0]) and torch.equal(counts.cpu(), want[2]) and int(live) == 64
    assert torch.isnan(losses).all() and (ids[6] == 32).all() and not gates[6].any() and int(ids[7, 0]) == 9
    d = fk.fk_route_backward(l, ids, counts, live, torch.ones((64, 4), device=DEV), torch.ones(2, device=DEV))
    keep = [r for r in range(64) if r not in (5, 6, 7)]
    assert torch.isfinite(d[keep]).all() and torch.isnan(d[5]).any()


def test_route_strided_logits_match_contiguous(gpu_lib):
    fk = gpu_lib
    for dtype, extra in ((torch.bfloat16, 8), (torch.float32, 3)):
        l = rand(300, 48, seed=2, dtype=dtype)
        a, b = fk.fk_route(l, 4), fk.fk_route(strided(l, extra), 4)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        dg = rand(300, 4, seed=3)
        assert torch.equal(fk.fk_route_backward(l, a[0], a[2], a[4], dg),
                           fk.fk_route_backward(strided(l, extra), a[0], a[2], a[4], dg))


# ---- products -------------------------------------------------------------------------

LINEAR_SIZES = [(1, 1, 1), (1, 64, 256), (3, 17, 40), (16, 130, 72), (17, 100, 515), (64, 256, 64), (130, 129, 128),
                (200, 384, 96), (257, 300, 1000), (300, 520, 33)]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("i", range(len(LINEAR_SIZES)))
def test_linear(gpu_lib, i, dtype):
    fk = gpu_lib
    M, N, K = LINEAR_SIZES[i]
    name = ACTS[i % len(ACTS)]
    log(f"linear {M} x {N} x {K} {dtype} {name}")
    X = rand(M, K, seed=i, dtype=dtype)
    Wt = rand(N, K, seed=i + 50, scale=K ** -0.5, dtype=dtype)
    b = rand(N, seed=i + 100, dtype=dtype)
    res = rand(M, N, seed=i + 150, dtype=dtype)
    y, z, e_y, e_z = R.linear(X, Wt, b, name, res)
    Y, pre = fk.fk_linear(X, Wt, b, act=name, residual=res, with_pre=True)
    check("Y", Y, y, e_y, dtype)
    check("pre", pre, z, e_z, dtype)
    dY = rand(M, N, seed=i + 200, dtype=dtype)
    kept = None if name == "none" else pre
    dx, dw, db, e_dx, e_dw, e_db = R.linear_grad(dY, X, Wt, name, kept)
    dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, act=name, pre=kept)
    check("dX", dX, dx, e_dx, dtype)
    check("dW", dW, dw, e_dw, dtype)
    check("dbias", dB, db, e_db, dtype)
    # plain, without bias and residual, and only what is asked for
    y, _, e_y, _ = R.linear(X, Wt, None, "none", None)
    Y, pre = fk.fk_linear(X, Wt)
    assert pre is None
    check("plain Y", Y, y, e_y, dtype)
    assert torch.equal(fk.fk_linear_backward(dY, X, Wt, act=name, pre=kept, with_dw=False, with_bias=False)[0], dX)
    assert torch.equal(fk.fk_linear_backward(dY, X, Wt, act=name, pre=kept, with_dx=False, with_bias=False)[1], dW)
    assert torch.equal(fk.fk_linear_backward(dY, X, Wt, act=name, pre=kept, with_dx=False, with_dw=False)[2], dB)


@pytest.mark.parametrize("M,N,K", [(1024, 2048, 256), (3100, 4104, 136), (2048, 1000, 2056), (130, 200, 9000), (40, 64, 16384)])
def test_linear_large_tiles_and_split_sums(gpu_lib, M, N, K):
    """Against float64 on the GPU: enough tiles for the 256-row ones, and few
    enough with a long sum for split ones."""
    fk = gpu_lib
    dtype = torch.bfloat16
    log(f"linear {M} x {N} x {K}")
    X, Wt = rand(M, K, seed=1, dtype=dtype), rand(N, K, seed=2, scale=K ** -0.5, dtype=dtype)
    b, dY = rand(N, seed=3, dtype=dtype), rand(M, N, seed=4, dtype=dtype)
    x, w, dy = X.double(), Wt.double(), dY.double()
    z = x @ w.t() + b.double()
    Y, pre = fk.fk_linear(X, Wt, b, act="silu", with_pre=True)
    e = (K + 24) * R.W * (x.abs() @ w.abs().t() + b.double().abs())
    check("pre", pre, z.cpu(), e.cpu(), dtype)
    check("Y", Y, (z * torch.sigmoid(z)).cpu(), (1.2 * e + 16 * R.W * z.abs()).cpu(), dtype)
    dX, dW, dB = fk.fk_linear_backward(dY, X, Wt)
    check("dX", dX, (dy @ w).cpu(), ((N + 24) * R.W * (dy.abs() @ w.abs())).cpu(), dtype)
    check("dW", dW, (dy.t() @ x).cpu(), ((M + 24) * R.W * (dy.abs().t() @ x.abs())).cpu(), dtype)
    check("dbias", dB, dy.sum(0).cpu(), ((M + 24) * R.W * dy.abs().sum(0)).cpu(), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_strides_and_fp32_outputs(gpu_lib, dtype):
    fk = gpu_lib
    M, N, K = 150, 88, 120
    for extra in (8, 3):
        X = strided(rand(M, K, seed=1, dtype=dtype), extra)
        Wt = strided(rand(N, K, seed=2, scale=K ** -0.5, dtype=dtype), extra)
        res = strided(rand(M, N, seed=3, dtype=dtype), extra)
        b = rand(N, seed=4)
        y, _, e_y, _ = R.linear(X, Wt, b, "gelu", res)
        Y, pre = fk.fk_linear(X, Wt, b, act="gelu", residual=res, out_dtype=torch.float32, with_pre=True)
        assert Y.dtype == torch.float32
        check("fp32 Y", Y, y, e_y, torch.float32)
        out = strided(torch.zeros((M, N), dtype=dtype, device=DEV), extra)
        fk.fk_linear(X, Wt, b, act="gelu", residual=res, Y=out)
        assert torch.isnan(out._base[:, N:]).all()
        check("strided Y", out, y, e_y, dtype)
        dY = strided(rand(M, N, seed=5), extra)  # fp32
        dx, dw, db, e_dx, e_dw, e_db = R.linear_grad(dY, X, Wt, "gelu", pre)
        dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, act="gelu", pre=pre, bias_dtype=torch.float32)
        check("dX", dX, dx, e_dx, dtype)
        check("dW", dW, dw, e_dw, dtype)
        check("dbias", dB, db, e_db, torch.float32)
    # the residual's own place
    res = res.contiguous()
    want, _ = fk.fk_linear(X, Wt, b, act="gelu", residual=res)
    got, _ = fk.fk_linear(X, Wt, b, act="gelu", residual=res, Y=res)
    assert got is res and torch.equal(got, want)


GROUPED = [  # T, share, E, N, K, loads, unrouted slots
    (1, 2, 4, 32, 64, "even", 0), (8, 2, 8, 130, 96, "even", 1), (40, 1, 3, 64, 200, "one", 0),
    (100, 2, 16, 72, 64, "even", 5), (300, 2, 5, 136, 130, "skew", 0), (150, 4, 70, 48, 40, "skew", 7),
    (600, 1, 2, 256, 64, "skew", 600), (513, 1, 4, 300, 72, "one", 2), (64, 3, 130, 40, 33, "even", 3)]


def _slots(M, E, loads, lost, seed):
    g = torch.Generator().manual_seed(seed)
    if loads == "even":
        ids = torch.randint(0, E, (M,), generator=g)
    elif loads == "one":
        ids = torch.full((M,), E - 1)
    else:
        ids = (E * torch.rand(M, generator=g) ** 3).long()
    if lost:
        ids[torch.randperm(M, generator=g)[:lost]] = E
    return ids.to(torch.int32).to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_linear(gpu_lib, case, dtype):
    fk = gpu_lib
    T, share, E, N, K, loads, lost = GROUPED[case]
    name = ("silu", "gelu", "none")[case % 3]
    M = T * share
    log(f"grouped {T} x {share} over {E}, {N} x {K} {dtype} {loads} lost={lost}")
    ids = _slots(M, E, loads, lost, case)
    slots, offsets = fk.fk_sort_inverse(ids, E + 1)
    X = rand(T, K, seed=case, dtype=dtype)
    Wt = rand(E, N, K, seed=case + 20, scale=K ** -0.5, dtype=dtype)
    b = rand(E, N, seed=case + 40, dtype=dtype)
    res = rand(M, N, seed=case + 60, dtype=dtype)
    where = {"slots": slots, "offsets": offsets, "share": share}
    y, z, e_y, e_z = R.linear(X, Wt, b, name, res, **where)
    Y, pre = fk.fk_linear(X, Wt, b, act=name, residual=res, with_pre=True, **where)
    check("Y", Y, y, e_y, dtype)
    check("pre", pre, z, e_z, dtype)
    assert not Y[(ids == E)].any()
    dY = rand(M, N, seed=case + 80, dtype=dtype)
    kept = None if name == "none" else pre
    dx, dw, db, e_dx, e_dw, e_db = R.linear_grad(dY, X, Wt, name, kept, **where)
    dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, act=name, pre=kept, **where)
    check("dX", dX, dx, e_dx, dtype)
    check("dW", dW, dw, e_dw, dtype)
    check("dbias", dB, db, e_db, dtype)
    if share == 1:
        # rows that lie in group order already: no slot list
        order = slots.long()
        Y2, _ = fk.fk_linear(X[order].contiguous(), Wt, b, act=name, residual=res[order].contiguous(), offsets=offsets)
        check("sorted Y", Y2, y[order.cpu()], e_y[order.cpu()], dtype)


def test_grouped_matches_plain_for_one_group(gpu_lib):
    fk = gpu_lib
    X, Wt = rand(700, 256, seed=1, dtype=torch.bfloat16), rand(512, 256, seed=2, dtype=torch.bfloat16)
    off = torch.tensor([0, 700], dtype=torch.int32, device=DEV)
    a, _ = fk.fk_linear(X, Wt, act="relu")
    b, _ = fk.fk_linear(X, Wt[None].contiguous(), act="relu", offsets=off)
    assert torch.equal(a, b)


def test_grouped_rows_past_32_bit_offsets(gpu_lib):
    """X and dY of more than 4 GB, rows taken from all over them by slots: a
    sample of rows against float64, dW of one group as a whole."""
    fk = gpu_lib
    T, K, N, E = 1_050_007, 2064, 128, 3
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, 100_000):
        X[i:i + 100_000].normal_(generator=g)
    assert X.numel() * 2 > 1 << 32
    Wt = rand(E, N, K, seed=2, scale=K ** -0.5, dtype=torch.bfloat16)
    ids = torch.randint(0, E + 1, (T,), generator=g, device=DEV, dtype=torch.int32)
    ids[-5:] = torch.tensor([0, 1, 2, 0, 1], dtype=torch.int32)
    slots, offsets = fk.fk_sort_inverse(ids, E + 1)
    where = {"slots": slots, "offsets": offsets}
    Y, _ = fk.fk_linear(X, Wt, **where)
    at = torch.cat((torch.arange(0, T, 30011, device=DEV), torch.arange(T - 5, T, device=DEV)))
    for e in range(E + 1):
        rows = at[ids[at] == e]
        x = X[rows].double()
        w = Wt[e].double() if e < E else torch.zeros((N, K), dtype=R.D, device=DEV)
        bound = (K + 24) * R.W * (x.abs() @ w.abs().t())
        check(f"Y of group {e}", Y[rows], (x @ w.t()).cpu(), bound.cpu(), torch.bfloat16)
    dY = rand(T, N, seed=5, dtype=torch.bfloat16)
    dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, **where)
    for e in range(E):
        rows = at[ids[at] == e]
        d, w = dY[rows].double(), Wt[e].double()
        check(f"dX of group {e}", dX[rows], (d @ w).cpu(), ((N + 24) * R.W * (d.abs() @ w.abs())).cpu(), torch.bfloat16)
    rows = (ids == 1).nonzero()[:, 0]
    want = torch.zeros((N, K), dtype=R.D, device=DEV)
    mag = torch.zeros((N, K), dtype=R.D, device=DEV)
    for part in rows.split(50_000):
        d, x = dY[part].double(), X[part].double()
        want += d.t() @ x
        mag += d.abs().t() @ x.abs()
    check("dW", dW[1], want.cpu(), ((rows.numel() + 24) * R.W * mag).cpu(), torch.bfloat16)
    assert not dX[ids == E].any()


# ---- combine -----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,d", [(1, 1, 1), (3, 2, 8), (5, 6, 100), (70, 8, 512), (33, 4, 2048), (9, 9, 2052),
                                      (4, 3, 4096), (3, 17, 8192), (2, 2, 10001), (500, 2, 16)])
def test_combine(gpu_lib, rows, k, d, dtype):
    fk = gpu_lib
    log(f"combine {rows} x {k} x {d} {dtype}")
    Y = rand(rows * k, d, seed=1, dtype=dtype)
    g = rand(rows, k, seed=2)
    res = strided(rand(rows, d, seed=3, dtype=dtype), 8)
    out, e = R.combine(Y, k, g, res)
    check("out", fk.fk_combine(Y, k, g, residual=res), out, e, dtype)
    out, e = R.combine(Y, k, None, None)
    check("plain sum", fk.fk_combine(Y, k), out, e, dtype)
    dOut = strided(rand(rows, d, seed=4, dtype=dtype), 16)
    dy, dg, e_dy, e_dg = R.combine_grad(dOut, Y, g)
    got = fk.fk_combine_backward(dOut, Y, g)
    check("dY", got[0], dy, e_dy, dtype)
    check("dgates", got[1], dg, e_dg, torch.float32)


def test_combine_skips_slots_without_gate(gpu_lib):
    fk = gpu_lib
    Y = rand(40, 96, seed=1, dtype=torch.bfloat16)
    g = rand(20, 2, seed=2)
    g[3, 1] = g[7, 0] = 0.0
    want = fk.fk_combine(torch.where((g.reshape(-1, 1) == 0).expand_as(Y), torch.zeros_like(Y), Y), 2, g)
    Y[7] = float("nan")
    Y[14] = float("inf")
    assert torch.equal(fk.fk_combine(Y, 2, g), want)
    dy, _ = fk.fk_combine_backward(torch.full((20, 96), float("inf"), dtype=torch.bfloat16, device=DEV), Y, g)
    assert not dy[7].any() and not dy[14].any()


# ---- gradients against differences ------------------------------------------------------------


def _slope(f, x, v, h=1e-5):
    """The derivative of f (64 bits) at x along v by central differences; its
    error is about h^2 third derivatives + 2^-52 / h, below 1e-8 here."""
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_gradients_against_differences(gpu_lib):
    """fp32 gradients along a random direction against central differences of
    the 64-bit forward functions, within the gradients' summed bounds."""
    fk = gpu_lib
    g = torch.Generator().manual_seed(5)

    def along(name, grad, bound, f, x):
        v = torch.randn(x.shape, generator=g, dtype=R.D)
        want = _slope(f, R.d64(x), v)
        got = (R.d64(grad) * v).sum()
        lim = R.SLACK * ((bound + R.W * R.d64(grad).abs()) * v.abs()).sum() + 1e-7 * (1 + want.abs())
        assert (got - want).abs() <= lim, f"{name}: {got} for {want}, {lim} allowed"

    X, w, b, dY = rand(6, 40, seed=1), rand(40, seed=2), rand(40, seed=3), rand(6, 40, seed=4)
    Y, mean, rstd = fk.fk_layer_norm(X, w, b)
    dX, dw, db = fk.fk_layer_norm_backward(dY, X, mean, rstd, w)
    bounds = R.layer_norm_grad(dY, X, w, 1e-5)[3:]
    along("norm dX", dX, bounds[0], lambda x: (R.layer_norm(x, w, b, 1e-5)[0] * R.d64(dY)).sum(), X)
    along("norm dw", dw, bounds[1], lambda x: (R.layer_norm(X, x, b, 1e-5)[0] * R.d64(dY)).sum(), w)
    along("norm db", db, bounds[2], lambda x: (R.layer_norm(X, w, x, 1e-5)[0] * R.d64(dY)).sum(), b)

    l, dg, dl = rand(30, 12, seed=5), rand(30, 3, seed=6), torch.tensor([0.5, 0.2], device=DEV)
    for norm in ("chosen", "all"):
        ids, gates, counts, losses, live = fk.fk_route(l, 3, norm=norm)
        d = fk.fk_route_backward(l, ids, counts, live, dg, dl, norm=norm)
        _, mag = R.route_grad(l, 3, norm, None, dg, dl)

        def total(x):
            r = R.route(x, 3, norm)
            return (r[1] * R.d64(dg)).sum() + (r[3] * R.d64(dl)).sum()
        along(f"route {norm}", d, 3 * P_REL * mag, total, l)

    X, Wt, b = rand(20, 24, seed=7), rand(3, 16, 24, seed=8, scale=0.2), rand(3, 16, seed=9)
    dY = rand(40, 16, seed=10)
    slots, offsets = fk.fk_sort_inverse(_slots(40, 3, "even", 4, 1), 4)
    where = {"slots": slots, "offsets": offsets, "share": 2}
    for name in ("gelu", "gelu_tanh", "silu"):
        _, pre = fk.fk_linear(X, Wt, b, act=name, with_pre=True, **where)
        dX, dW, dB = fk.fk_linear_backward(dY, X, Wt, act=name, pre=pre, **where)
        _, _, _, e_dx, e_dw, e_db = R.linear_grad(dY, X, Wt, name, pre, **where)
        # the kept pre-activations are off by their own bound, which the slopes pass on
        off = 1 + 200 * 24
        dsum = fk.fk_combine(dX, 2)
        e_dx = e_dx.view(20, 2, 24).sum(1)
        f = lambda x, w_, b_: (R.linear(x, w_, b_, name, None, **where)[0] * R.d64(dY)).sum()  # noqa: E731
        along(f"{name} dX", dsum, e_dx + off * R.W * R.d64(dsum).abs().mean(), lambda x: f(x, Wt, b), X)
        along(f"{name} dW", dW, e_dw + off * R.W * R.d64(dW).abs().mean(), lambda x: f(X, x, b), Wt)
        along(f"{name} db", dB, e_db + off * R.W * R.d64(dB).abs().mean(), lambda x: f(X, Wt, x), b)

    Y, gt, do = rand(24, 20, seed=11), rand(8, 3, seed=12), rand(8, 20, seed=13)
    dY, dgt = fk.fk_combine_backward(do, Y, gt)
    _, _, e_dy, e_dg = R.combine_grad(do, Y, gt)
    along("combine dY", dY, e_dy, lambda x: (R.combine(x, 3, gt, None)[0] * R.d64(do)).sum(), Y)
    along("combine dgates", dgt, e_dg, lambda x: (R.combine(Y, 3, x, None)[0] * R.d64(do)).sum(), gt)


# ---- streams, graphs, repeatability ----------------------------------------------------------


def _block(fk, X, p):
    """A routed block's forward and backward pass; every result."""
    T, d = X.shape
    E, k = p["up"].shape[0], 2
    h, mean, rstd = fk.fk_layer_norm(X, p["w"], p["b"])
    logits, _ = fk.fk_linear(h, p["router"], out_dtype=torch.float32)
    ids, gates, counts, losses, live = fk.fk_route(logits, k)
    slots, offsets = fk.fk_sort_inverse(ids.view(-1), E + 1)
    where = {"slots": slots, "offsets": offsets}
    a, pre = fk.fk_linear(h, p["up"], p["ub"], act="silu", with_pre=True, share=k, **where)
    y, _ = fk.fk_linear(a, p["down"], **where)
    out = fk.fk_combine(y, k, gates, residual=X)
    dy, dgates = fk.fk_combine_backward(out, y, gates)
    da, ddown, _ = fk.fk_linear_backward(dy, a, p["down"], **where)
    dh, dup, dub = fk.fk_linear_backward(da, h, p["up"], act="silu", pre=pre, share=k, **where)
    dl = fk.fk_route_backward(logits, ids, counts, live, dgates, p["dl"])
    dh2, drouter, _ = fk.fk_linear_backward(dl, h, p["router"])
    dX, dw, db = fk.fk_layer_norm_backward(fk.fk_combine(dh, k, residual=dh2), X, mean, rstd, p["w"])
    return [h, logits, ids, gates, counts, losses, out, ddown, dup, dub, drouter, dX, dw, db]


def _block_params(E, d, hid, dtype):
    return {"w": rand(d, seed=1, shift=1.0, scale=0.1, dtype=dtype), "b": rand(d, seed=2, dtype=dtype),
            "router": rand(E, d, seed=3, scale=d ** -0.5, dtype=dtype),
            "up": rand(E, hid, d, seed=4, scale=d ** -0.5, dtype=dtype), "ub": rand(E, hid, seed=5, dtype=dtype),
            "down": rand(E, d, hid, seed=6, scale=hid ** -0.5, dtype=dtype),
            "dl": torch.tensor([0.01, 0.001], device=DEV)}


def test_block_repeats_bitwise_and_runs_on_another_stream(gpu_lib):
    fk = gpu_lib
    p = _block_params(8, 256, 320, torch.bfloat16)
    X = rand(777, 256, seed=9, dtype=torch.bfloat16)
    want = _block(fk, X, p)
    assert all(torch.isfinite(t.float()).all() for t in want)
    again = _block(fk, X, p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = _block(fk, X, p)
    torch.cuda.synchronize()
    for u, v, w in zip(want, again, other):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_block_in_a_graph(gpu_lib):
    """Captured once, replayed over changed inputs, each replay equal to the
    eager result, with eager work between the replays."""
    fk = gpu_lib
    p = _block_params(4, 128, 192, torch.bfloat16)
    X = rand(130, 128, seed=9, dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _block(fk, X, p)  # sizes the stream's workspace
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = _block(fk, X, p)
    for seed in (9, 10, 11, 9):
        X.copy_(rand(130, 128, seed=seed, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want = _block(fk, X.clone(), p)
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)


def test_refusals_of_the_binding(gpu_lib):
    fk = gpu_lib
    X = rand(8, 32, seed=1)
    Wt = rand(16, 32, seed=2)
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        fk.fk_layer_norm(X.cpu())
    with pytest.raises(ValueError):
        fk.fk_layer_norm(X.double())
    with pytest.raises(ValueError):
        fk.fk_layer_norm(X.t())
    with pytest.raises(ValueError):
        fk.fk_layer_norm(X, weight=X[0, :5])
    with pytest.raises(fk.FkError):
        fk.fk_layer_norm(X, eps=-1.0)
    with pytest.raises(fk.FkError):
        fk.fk_layer_norm(X[:4], Y=X.view(-1)[16:16 + 128].view(4, 32))
    with pytest.raises(fk.FkError):
        fk.fk_route(X, 33)
    with pytest.raises(ValueError):
        fk.fk_route(X, 2, norm="none")
    with pytest.raises(ValueError):
        fk.fk_route(X, 2, valid=torch.ones(7, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError):
        fk.fk_linear(X, Wt[:, :31])
    with pytest.raises(ValueError):
        fk.fk_linear(X, Wt, act="swish")
    with pytest.raises(ValueError):
        fk.fk_linear(X, Wt, slots=off)
    with pytest.raises(ValueError):
        fk.fk_linear(X, Wt[None], offsets=off[:1])
    with pytest.raises(fk.FkError):
        fk.fk_linear(X, Wt[None], offsets=off, share=2)   # no slot list to share rows by
    with pytest.raises(fk.FkError):
        fk.fk_linear(X, Wt, Y=X[:, :16])                 # output over an input
    with pytest.raises(fk.FkError):
        fk.fk_linear(X.view(-1)[1:225].view(7, 32), Wt)   # not on 16 bytes
    with pytest.raises(ValueError):
        fk.fk_linear_backward(rand(8, 16, seed=3), X, Wt, act="gelu")
    with pytest.raises(ValueError):
        fk.fk_combine(X, 3)
    with pytest.raises(fk.FkError):
        fk.fk_combine(rand(130, 4, seed=1), 65)  # more slots a row than there may be
