"""Plain 64-bit implementations of the expert-block operators (numpy-like torch
code on the CPU), and the bounds that the GPU's results are held to.

Bounds.  u is the unit roundoff of an output's type (2^-24, 2^-8 for bf16,
2^-11 for fp16); w = 2^-24 that of the fp32 arithmetic inside.  A sum of n
terms in fp32, in whatever order, is within n w of the sum of their absolute
values (first order), so every bound below is u |result| plus w times the
number of roundings on the way times the absolute values that they act on.
SLACK = 1.25 covers the second-order terms.  fp16 results below its smallest
normal number round by half of 2^-24 (TINY).
"""
import math

import torch

D = torch.float64
W = 2.0 ** -24
U = {D: 2.0 ** -53, torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {D: 0.0, torch.float32: 1e-38, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}
SLACK = 1.25


def d64(t):
    return t.detach().to("cpu").to(D)


def check(name, got, want, bound, dtype):
    """|got - want| <= bound + u |want| elementwise; non-finite values must agree."""
    got = d64(got)
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} for {tuple(want.shape)}"
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN in other places"
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), f"{name}: infinities differ"
    err = (got - want).abs()
    lim = SLACK * (bound + U[dtype] * want.abs()) + TINY[dtype]
    bad = fin & ~(err <= lim)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {got[i]:.9g} for "
                             f"{want[i]:.9g}, off by {err[i]:.3g}, {lim[i]:.3g} allowed")


# ---- layer norm ----------------------------------------------------------------


def norm_depth(d):
    """Roundings a term meets in a row's sum: those of one thread (at most 32
    elements, or d / 256 of a long row), the lanes' and the waves'."""
    return (32 if d <= 8192 else math.ceil(d / 256)) + 12


def layer_norm(X, w, b, eps):
    """y, mean, rstd and the bounds of y, mean, xh, and rstd (relative)."""
    x = d64(X)
    d = x.shape[1]
    wt = torch.ones(d, dtype=D) if w is None else d64(w)
    bt = torch.zeros(d, dtype=D) if b is None else d64(b)
    mu = x.mean(1, keepdim=True)
    xc = x - mu
    var = (xc * xc).mean(1, keepdim=True)
    r = (var + eps) ** -0.5
    xh = xc * r
    y = xh * wt + bt
    n = norm_depth(d)
    e_mu = n * W * x.abs().mean(1, keepdim=True)
    e_xc = e_mu + W * xc.abs()
    # the variance around a mean that is off by e is larger by e^2
    e_var = (n + 2) * W * var + 2 * (e_xc * xc.abs()).mean(1, keepdim=True) + (e_xc ** 2).mean(1, keepdim=True)
    rel_r = 0.5 * e_var / (var + eps) + 4 * W
    e_xh = r * e_xc + xh.abs() * (rel_r + W)
    e_y = wt.abs() * e_xh + 2 * W * ((xh * wt).abs() + bt.abs())
    return y, mu[:, 0], r[:, 0], e_y, e_mu[:, 0], e_xh, rel_r[:, 0]


def layer_norm_grad(dY, X, w, eps):
    """dx, dw, db and their bounds (mean and rstd as the forward pass gives them)."""
    _, mu, r, _, _, e_xh, rel_r = layer_norm(X, None, None, eps)
    x, dy = d64(X), d64(dY)
    rows, d = x.shape
    wt = torch.ones(d, dtype=D) if w is None else d64(w)
    r, rel_r = r[:, None], rel_r[:, None]
    xh = (x - mu[:, None]) * r
    g = dy * wt
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    n = norm_depth(d)
    e_c1 = (n + 1) * W * g.abs().mean(1, keepdim=True)
    e_c2 = (n + 2) * W * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * e_xh).mean(1, keepdim=True)
    mag = g.abs() + c1.abs() + (xh * c2).abs()
    e_dx = r * (5 * W * mag + e_c1 + xh.abs() * e_c2 + e_xh * c2.abs()) + rel_r * r * (g - c1 - xh * c2).abs()
    dw, db = (dy * xh).sum(0), dy.sum(0)
    m = rows + 30
    e_dw = (m * W * (dy * xh).abs() + dy.abs() * e_xh).sum(0)
    e_db = m * W * dy.abs().sum(0)
    return dx, dw, db, e_dx, e_dw, e_db


# ---- router ---------------------------------------------------------------------


def route(logits, k, norm, valid=None):
    """ids, gates, counts, losses, n and p (rows left out are zero)."""
    l = d64(logits)
    T, E = l.shape
    live = (l > -math.inf).any(1) | torch.isnan(l).any(1)
    if valid is not None:
        live &= valid.to("cpu").bool()
    on = live[:, None]
    key = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l)
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    val = key.gather(1, order)
    has = on & (val > -math.inf)
    ids = torch.where(has, order, torch.full_like(order, E))
    lz = torch.where(on, l, torch.zeros_like(l))
    # differences from the row's largest, which a log of the sum added to a
    # huge logit would lose
    m = torch.where(on, key.max(1, keepdim=True)[0], torch.zeros_like(l[:, :1]))
    e = torch.exp(lz - m)
    lse = m[:, 0] + torch.log(e.sum(1))
    p = torch.where(on, e / e.sum(1, keepdim=True), torch.zeros_like(l))
    ge = torch.where(has, torch.exp(torch.where(has, val, m) - m), torch.zeros_like(val))
    if norm == "chosen":
        s = ge.sum(1, keepdim=True)
    else:
        s = e.sum(1, keepdim=True)
    gates = torch.where(has, ge / s, torch.zeros_like(val))
    counts = torch.bincount(ids.reshape(-1), minlength=E + 1)[:E]
    n = max(1, int(live.sum()))
    f = counts.to(D) / max(1, int(counts.sum()))
    losses = torch.stack((E * (f * p.sum(0)).sum() / n, torch.where(live, lse * lse, 0 * lse).sum() / n))
    return ids.to(torch.int32), gates, counts.to(torch.int32), losses, int(live.sum()), p, lse, live, f


def route_grad(logits, k, norm, valid, d_gates, d_losses):
    """d_logits and the absolute values that its roundings act on."""
    ids, gates, counts, _, n, p, lse, live, f = route(logits, k, norm, valid)
    T, E = p.shape
    n = max(1, n)
    dbal, dz = (0.0, 0.0) if d_losses is None else d64(d_losses).tolist()
    dg = torch.zeros((T, k), dtype=D) if d_gates is None else d64(d_gates)
    dg = torch.where(ids < E, dg, torch.zeros_like(dg))
    v = dbal * E / n * f
    pv = (p * v).sum(1, keepdim=True)
    zt = 2 * dz * torch.where(live, lse, 0 * lse)[:, None] / n
    dl = p * (v - pv + zt)
    mag = p * (v.abs() + (p * v.abs()).sum(1, keepdim=True) + zt.abs())
    at = ids.long().clamp_max(E - 1)
    inner = (gates * dg).sum(1, keepdim=True)
    ainner = (gates * dg.abs()).sum(1, keepdim=True)
    if norm == "chosen":
        dl = dl.scatter_add(1, at, gates * (dg - inner))
        mag = mag.scatter_add(1, at, gates * (dg.abs() + ainner))
    else:
        dl = dl.scatter_add(1, at, gates * dg) - p * inner
        mag = mag.scatter_add(1, at, gates * dg.abs()) + p * ainner
    return dl, mag


# ---- products ----------------------------------------------------------------------


def act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(act(name, z).sum(), z)[0]


def groups_of(M, offsets, slots, G, share):
    """(group, slots, rows of X) of every group; one of everything without offsets."""
    if offsets is None:
        yield 0, torch.arange(M), torch.arange(M)
        return
    o = offsets.cpu().tolist()
    s = torch.arange(M) if slots is None else slots.cpu().long()
    for g in range(G):
        mine = s[o[g]:o[g + 1]]
        yield g, mine, mine // share


def linear(X, Wt, bias, name, residual, slots=None, offsets=None, share=1):
    """Y, pre and their bounds."""
    x, w = d64(X), d64(Wt)
    grouped = offsets is not None
    G = w.shape[0] if grouped else 1
    N, K = w.shape[-2:]
    M = x.shape[0] * share
    z, e, y = (torch.zeros((M, N), dtype=D) for _ in range(3))
    for g, sl, rw in groups_of(M, offsets, slots, G, share):
        wg = w[g] if grouped else w
        b = torch.zeros(N, dtype=D) if bias is None else d64(bias[g] if grouped else bias)
        z[sl] = x[rw] @ wg.t() + b
        e[sl] = (K + 24) * W * (x[rw].abs() @ wg.abs().t() + b.abs())
        y[sl] = act(name, z[sl])
        if residual is not None:
            y[sl] += d64(residual)[sl]
    # an activation's slope is below 1.2; its own roundings act on |z|
    e_y = 1.2 * e + 16 * W * z.abs()
    if residual is not None:
        e_y = e_y + W * d64(residual).abs()
    return y, z, e_y, e


def linear_grad(dY, X, Wt, name, pre, slots=None, offsets=None, share=1):
    """dX, dW, db and their bounds."""
    x, w, dy = d64(X), d64(Wt), d64(dY)
    u = U[X.dtype]
    grouped = offsets is not None
    G = w.shape[0] if grouped else 1
    N, K = w.shape[-2:]
    M = dy.shape[0]
    slope = torch.ones_like(dy) if pre is None else act_slope(name, d64(pre))
    dz = dy * slope
    # the slope's roundings act on its terms: 1 and |z| for the smooth ones
    e_dz = torch.zeros_like(dz)
    if pre is not None and name not in ("none", "relu"):
        e_dz = 24 * W * dy.abs() * (1 + d64(pre).abs())
    plain = name == "none" and dY.dtype == X.dtype  # dY goes in as it is
    r_dz = e_dz + (0 if plain else u * (dz.abs() + e_dz)) + (0 if plain else TINY[X.dtype])
    dx, e_dx = torch.zeros((M, K), dtype=D), torch.zeros((M, K), dtype=D)
    dw, e_dw = torch.zeros((G, N, K), dtype=D), torch.zeros((G, N, K), dtype=D)
    db, e_db = torch.zeros((G, N), dtype=D), torch.zeros((G, N), dtype=D)
    for g, sl, rw in groups_of(M, offsets, slots, G, share):
        wg = w[g] if grouped else w
        a = dz[sl].abs()
        dx[sl] = dz[sl] @ wg
        e_dx[sl] = (N + 24) * W * (a @ wg.abs()) + r_dz[sl] @ wg.abs()
        dw[g] = dz[sl].t() @ x[rw]
        m = len(sl) + 24
        e_dw[g] = m * W * (a.t() @ x[rw].abs()) + r_dz[sl].t() @ x[rw].abs()
        db[g] = dz[sl].sum(0)
        e_db[g] = (m * W * a + e_dz[sl] + W * a).sum(0)
    if not grouped:
        dw, e_dw, db, e_db = dw[0], e_dw[0], db[0], e_db[0]
    return dx, dw, db, e_dx, e_dw, e_db


# ---- combine -----------------------------------------------------------------------


def combine(Y, k, gates, residual):
    y = d64(Y)
    rows, d = y.shape[0] // k, y.shape[1]
    y = y.view(rows, k, d)
    g = torch.ones((rows, k), dtype=D) if gates is None else d64(gates)
    t = torch.where(g[:, :, None] == 0, torch.zeros_like(y), y * g[:, :, None])
    out, mag = t.sum(1), t.abs().sum(1)
    if residual is not None:
        out, mag = out + d64(residual), mag + d64(residual).abs()
    return out, (k + 2) * W * mag


def combine_grad(dOut, Y, gates):
    do, y, g = d64(dOut), d64(Y), d64(gates)
    rows, d = do.shape
    k = g.shape[1]
    dy = (g[:, :, None] * do[:, None]).view(rows * k, d)
    t = y.view(rows, k, d) * do[:, None]
    return dy, t.sum(2), W * dy.abs(), (norm_depth(d) + 1) * W * t.abs().sum(2)
