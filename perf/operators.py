"""The expert-block operators and the cases they are measured on.

A block routes rows to experts: layer norm, router with its balance loss, the
experts' products over slots sorted by expert, and the weighted sum of every
row's expert outputs.  Each operator is given here in its plain form
(elementary torch operations in 32 bits, rounded once at the end), as the call
a user makes of the library (`own` true), and by its definition in 64 bits
(`exact`).

  norm      layer norm over the last dimension, forward or forward + backward
  route     top-k router with per-expert counts, balance and z losses
  linear    act(X W^T + b) + R, one weight matrix
  experts   the same with one weight matrix per expert, rows given by a slot
            list sorted by expert (slot s = row * share + j)
  combine   out[t] = R[t] + sum_j gate[t, j] Y[t k + j]
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # a handful of rows while tokens are produced one by one: latency
        {"name": "norm_token", "op": "norm", "dir": "fwd", "dtype": "bf16", "rows": 4, "d": 4096},
        # a training step's rows, an odd number of them
        {"name": "norm_train", "op": "norm", "dir": "train", "dtype": "bf16", "rows": 32749, "d": 4096},
        # routing of the rows of one decoding step
        {"name": "route_token", "op": "route", "dir": "fwd", "dtype": "fp32", "rows": 16, "experts": 64, "k": 6,
         "norm": "chosen", "padded": 0.0, "masked": 0.0},
        # routing of a large training batch with padding and masked experts
        {"name": "route_train", "op": "route", "dir": "train", "dtype": "fp32", "rows": 262144, "experts": 128, "k": 8,
         "norm": "chosen", "padded": 0.1, "masked": 0.02},
        # one token through an up projection: a stream of the weights
        {"name": "linear_token", "op": "linear", "dir": "fwd", "dtype": "bf16", "rows": 1, "n": 16384, "k_in": 4096,
         "act": "gelu", "residual": False},
        # a long prompt through a projection with everything in its epilogue
        {"name": "linear_prompt", "op": "linear", "dir": "fwd", "dtype": "bf16", "rows": 16384, "n": 8192,
         "k_in": 4096, "act": "gelu", "residual": True},
        # the gradients of a training step's projection
        {"name": "linear_train", "op": "linear", "dir": "bwd", "dtype": "bf16", "rows": 16384, "n": 4096,
         "k_in": 4096, "act": "gelu_tanh", "residual": False},
        # embeddings in fp32 through an odd-sized head
        {"name": "linear_odd", "op": "linear", "dir": "fwd", "dtype": "fp32", "rows": 5003, "n": 1001, "k_in": 769,
         "act": "silu", "residual": True},
        # one decoding step of 32 sequences: a few rows for each of many experts
        {"name": "experts_token", "op": "experts", "dir": "fwd", "dtype": "bf16", "rows": 32, "share": 2,
         "experts": 64, "skew": 0.3, "n": 4096, "k_in": 2048, "act": "silu"},
        # the gradients of a training step's experts, unevenly loaded
        {"name": "experts_train", "op": "experts", "dir": "bwd", "dtype": "bf16", "rows": 16381, "share": 2,
         "experts": 32, "skew": 0.5, "n": 4096, "k_in": 2048, "act": "silu"},
        # the sum of a decoding step's expert rows
        {"name": "combine_token", "op": "combine", "dir": "fwd", "dtype": "bf16", "rows": 8, "d": 4096, "k": 6,
         "residual": True},
        # the sum and its gradients over a training batch
        {"name": "combine_train", "op": "combine", "dir": "train", "dtype": "bf16", "rows": 16411, "d": 4096, "k": 4,
         "residual": True},
    ]


def _span(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: a multiple of 64, of 8, or any number."""
    v, m = _span(rng, lo, hi), rng.choice((64, 64, 8, 1))
    return max(lo, v // m * m)


def draw(rng):
    op = rng.choice(("norm", "route", "linear", "linear", "experts", "experts", "combine"))
    c = {"op": op, "dir": "fwd", "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
    if op == "norm":
        c["dir"] = rng.choice(("fwd", "train"))
        c["d"] = _width(rng, 64, 8192)
        c["rows"] = _span(rng, 1, min(1 << 18, (1 << 26) // c["d"]))
    elif op == "route":
        c["dir"] = rng.choice(("fwd", "train"))
        c["experts"] = rng.choice((8, 16, 32, 60, 64, 128, 160, 256))
        c["k"] = rng.choice((1, 2, 4, 6, 8))
        c["rows"] = _span(rng, 1, (1 << 25) // c["experts"])
        c["norm"] = rng.choice(("chosen", "all"))
        c["padded"] = rng.choice((0.0, 0.1, 0.3))
        c["masked"] = rng.choice((0.0, 0.02))
    elif op == "linear":
        c["dir"] = rng.choice(("fwd", "bwd"))
        c["n"] = _width(rng, 128, 16384)
        c["k_in"] = _width(rng, 128, 4096)
        c["rows"] = _span(rng, 1, min(16384, (1 << 38) // (c["n"] * c["k_in"])))
        c["act"] = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
        c["residual"] = c["dir"] == "fwd" and rng.random() < 0.5
    elif op == "experts":
        c["dir"] = rng.choice(("fwd", "bwd"))
        c["experts"] = rng.choice((4, 8, 16, 32, 64))
        c["share"] = rng.choice((1, 2, 4))
        c["rows"] = _span(rng, 1, 32768 // c["share"])
        c["skew"] = rng.choice((0.0, 0.3, 0.5))
        c["n"] = _width(rng, 128, 4096)
        c["k_in"] = _width(rng, 128, 2048)
        c["act"] = rng.choice(("none", "gelu", "silu"))
    else:
        c["dir"] = rng.choice(("fwd", "train"))
        c["d"] = _width(rng, 64, 8192)
        c["k"] = rng.choice((1, 2, 4, 6, 8))
        c["rows"] = _span(rng, 1, max(1, (1 << 26) // (c["d"] * c["k"])))
        c["residual"] = rng.random() < 0.5
    return c


def _shares(case):
    """How the experts' loads are spread: a power law of their rank."""
    w = [(e + 1.0) ** -case["skew"] for e in range(case["experts"])]
    s = sum(w)
    return [x / s for x in w]


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev)

    s = {"case": case}
    rows = case["rows"]
    if case["op"] == "norm":
        d = case["d"]
        # residual-stream rows: a common offset and a few columns much larger than the rest
        col = torch.where(uniform(d) < 0.01, 10.0, 1.0)
        s["X"] = (torch.randn((rows, d), generator=g, device=dev) * col + 0.3).to(dt)
        s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dt)
        s["bias"] = normal(d, scale=0.1)
        if case["dir"] != "fwd":
            s["dY"] = normal(rows, d)
    elif case["op"] == "route":
        E, k = case["experts"], case["k"]
        s["logits"] = normal(rows, E, scale=1.5)
        if case["masked"]:
            s["logits"].masked_fill_(uniform(rows, E) < case["masked"], -math.inf)
        s["valid"] = uniform(rows) >= case["padded"] if case["padded"] else None
        if case["dir"] != "fwd":
            s["d_gates"] = normal(rows, k, dtype=torch.float32, scale=1.0 / rows)
            s["d_losses"] = torch.tensor([0.01, 0.001], device=dev)
    elif case["op"] in ("linear", "experts"):
        N, K = case["n"], case["k_in"]
        lead = () if case["op"] == "linear" else (case["experts"],)
        M = rows * case.get("share", 1)
        s["X"] = normal(rows, K)
        s["W"] = normal(*lead, N, K, scale=K ** -0.5)
        s["bias"] = normal(*lead, N, scale=0.1)
        s["residual"] = normal(M, N) if case.get("residual") else None
        if case["op"] == "experts":
            # every row picks `share` different experts, the loads following a power law
            w = torch.tensor(_shares(case), device=dev)
            score = torch.log(w) - torch.log(-torch.log(uniform(rows, case["experts"]).clamp(1e-7, 1 - 1e-7)))
            ids = torch.sort(score, dim=1, descending=True, stable=True)[1][:, : case["share"]].reshape(-1)
            _, slots = torch.sort(ids, stable=True)
            counts = torch.bincount(ids, minlength=case["experts"])
            s["slots"] = slots.to(torch.int32)
            s["offsets"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
            s["ids"] = ids  # the expert of every slot
            s["capacity"] = int(counts.max())
        if case["dir"] != "fwd":
            s["dY"] = normal(M, N)
            s["pre"] = normal(M, N)  # the pre-activations kept by the forward pass
    else:
        d, k = case["d"], case["k"]
        s["Y"] = normal(rows * k, d)
        gates = uniform(rows, k) + 0.05
        s["gates"] = gates / gates.sum(1, keepdim=True)
        s["residual"] = normal(rows, d) if case["residual"] else None
        if case["dir"] != "fwd":
            s["dOut"] = normal(rows, d)
    return s


# ---- the formulas, for 32 and 64 bits ------------------------------------------


def _act(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _norm(s):
    dt = s["X"].dtype
    x, w, b = s["X"].float(), s["weight"].float(), s["bias"].float()
    mu = x.mean(1, keepdim=True)
    xc = x - mu
    r = torch.rsqrt((xc * xc).mean(1, keepdim=True) + 1e-5)
    xh = xc * r
    y = (xh * w + b).to(dt)
    if s["case"]["dir"] == "fwd":
        return {"Y": y, "mean": mu[:, 0], "rstd": r[:, 0]}
    dy = s["dY"].float()
    g = dy * w
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"Y": y, "dX": dx.to(dt), "dweight": (dy * xh).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}


def _route(s):
    c = s["case"]
    l = s["logits"].float()
    T, E, k = c["rows"], c["experts"], c["k"]
    top = l.max(1, keepdim=True)[0]
    live = top[:, 0] != -math.inf
    if s["valid"] is not None:
        live = live & s["valid"]
    on = live[:, None]
    m = torch.where(on, top, torch.zeros_like(top))
    e = torch.where(on, torch.exp(l - m), torch.zeros_like(l))
    tot = torch.where(on, e.sum(1, keepdim=True), torch.ones_like(m))
    p = e / tot
    lse = torch.where(on, m + torch.log(tot), torch.zeros_like(m))
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    has = on & (val != -math.inf)
    ids = torch.where(has, idx, torch.full_like(idx, E))
    if c["norm"] == "chosen":
        ge = torch.where(has, torch.exp(val - m), torch.zeros_like(val))
        gates = ge / torch.where(on, ge.sum(1, keepdim=True), torch.ones_like(m))
    else:
        gates = torch.where(has, p.gather(1, idx), torch.zeros_like(val))
    counts = torch.bincount(ids.reshape(-1), minlength=E + 1)[:E]
    n = live.sum().clamp_min(1).float()
    f = counts.float() / counts.sum().clamp_min(1).float()
    balance = E * (f * (p.sum(0) / n)).sum()
    z = (lse * lse).sum() / n
    out = {"ids": ids.to(torch.int32), "gates": gates, "counts": counts.to(torch.int32),
           "losses": torch.stack((balance, z))}
    if c["dir"] == "fwd":
        return out
    dg, (dbal, dz) = s["d_gates"], s["d_losses"]
    v = dbal * E / n * f
    dl = p * (v - (p * v).sum(1, keepdim=True)) + dz * 2 / n * lse * p
    dg = torch.where(has, dg, torch.zeros_like(dg))
    inner = (gates * dg).sum(1, keepdim=True)
    if c["norm"] == "chosen":
        dl = dl.scatter_add(1, idx, gates * (dg - inner))
    else:
        dl = (dl - p * inner).scatter_add(1, idx, gates * dg)
    out["d_logits"] = dl.to(s["logits"].dtype)
    return out


def _linear(s):
    c, dt = s["case"], s["X"].dtype
    x, w, b = s["X"].float(), s["W"].float(), s["bias"].float()
    if c["dir"] == "fwd":
        y = _act(c["act"], x @ w.t() + b)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"Y": y.to(dt)}
    dz = s["dY"].float() * _act_slope(c["act"], s["pre"].float())
    return {"dX": (dz @ w).to(dt), "dW": (dz.t() @ x).to(dt), "dbias": dz.sum(0).to(dt)}


def _experts(s):
    """Every expert's rows in a block of as many rows as the fullest one has."""
    c, dt = s["case"], s["X"].dtype
    w, b = s["W"].float(), s["bias"].float()
    slots = s["slots"].long()
    e = s["ids"][slots]
    at = torch.arange(slots.numel(), device=slots.device) - s["offsets"].long()[e]
    x = s["X"].float()
    xp = x.new_zeros((c["experts"], s["capacity"], c["k_in"]))
    xp[e, at] = x[slots // c["share"]]
    if c["dir"] == "fwd":
        y = _act(c["act"], torch.bmm(xp, w.transpose(1, 2).contiguous()) + b[:, None])
        out = x.new_empty((slots.numel(), c["n"]))
        out[slots] = y[e, at]
        return {"Y": out.to(dt)}
    dz = s["dY"].float() * _act_slope(c["act"], s["pre"].float())
    dzp = x.new_zeros((c["experts"], s["capacity"], c["n"]))
    dzp[e, at] = dz[slots]
    dx = x.new_empty((slots.numel(), c["k_in"]))
    dx[slots] = torch.bmm(dzp, w)[e, at]
    dw = torch.bmm(dzp.transpose(1, 2).contiguous(), xp)
    return {"dX": dx.to(dt), "dW": dw.to(dt), "dbias": dzp.sum(1).to(dt)}


def _combine(s):
    c, dt = s["case"], s["Y"].dtype
    y, g = s["Y"].float().view(c["rows"], c["k"], c["d"]), s["gates"]
    out = (y * g[:, :, None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    if c["dir"] == "fwd":
        return {"out": out.to(dt)}
    do = s["dOut"].float()
    dy = (g[:, :, None] * do[:, None]).view(c["rows"] * c["k"], c["d"])
    return {"out": out.to(dt), "dY": dy.to(dt), "dgates": (y * do[:, None]).sum(2)}


PLAIN = {"norm": _norm, "route": _route, "linear": _linear, "experts": _experts, "combine": _combine}


def _called(s):
    """The same passes as calls of the library."""
    import exact_lloyd_means_flashassign_amd as fk
    c = s["case"]
    op, fwd = c["op"], c["dir"] == "fwd"
    if op == "norm":
        y, mean, rstd = fk.fk_layer_norm(s["X"], s["weight"], s["bias"], eps=1e-5)
        if fwd:
            return {"Y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = fk.fk_layer_norm_backward(s["dY"], s["X"], mean, rstd, s["weight"])
        return {"Y": y, "dX": dx, "dweight": dw, "dbias": db}
    if op == "route":
        ids, gates, counts, losses, live = fk.fk_route(s["logits"], c["k"], norm=c["norm"], valid=s["valid"])
        out = {"ids": ids, "gates": gates, "counts": counts, "losses": losses}
        if not fwd:
            out["d_logits"] = fk.fk_route_backward(s["logits"], ids, counts, live, s["d_gates"], s["d_losses"],
                                                   norm=c["norm"], valid=s["valid"])
        return out
    if op in ("linear", "experts"):
        where = {"slots": s["slots"], "offsets": s["offsets"], "share": c["share"]} if op == "experts" else {}
        if fwd:
            return {"Y": fk.fk_linear(s["X"], s["W"], s["bias"], act=c["act"], residual=s["residual"], **where)[0]}
        dx, dw, db = fk.fk_linear_backward(s["dY"], s["X"], s["W"], act=c["act"], pre=s["pre"], **where)
        return {"dX": dx, "dW": dw, "dbias": db}
    out = fk.fk_combine(s["Y"], c["k"], s["gates"], residual=s["residual"])
    if fwd:
        return {"out": out}
    dy, dg = fk.fk_combine_backward(s["dOut"], s["Y"], s["gates"])
    return {"out": out, "dY": dy, "dgates": dg}


def run(state):
    return _called(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    b, rows = SIZE[case["dtype"]], case["rows"]
    fwd = case["dir"] == "fwd"
    if case["op"] == "norm":
        d = case["d"]
        if fwd:
            return {"bytes": b * (2 * rows * d + 2 * d) + 8 * rows, "flops": 8 * rows * d}
        # forward and backward: x, dy read, y, dx written (x once for both)
        return {"bytes": b * (4 * rows * d + 4 * d), "flops": 20 * rows * d}
    if case["op"] == "route":
        E, k = case["experts"], case["k"]
        bytes_ = b * rows * E + 8 * rows * k + 4 * E
        if case["padded"]:
            bytes_ += rows
        if not fwd:
            bytes_ += b * rows * E + 4 * rows * k
        return {"bytes": bytes_, "flops": (8 if fwd else 16) * rows * E}
    if case["op"] in ("linear", "experts"):
        N, K, share = case["n"], case["k_in"], case.get("share", 1)
        M, used, G = rows * share, 1.0, 1
        if case["op"] == "experts":
            G = case["experts"]
            # the experts that some row is expected to reach
            used = min(sum(1 - (1 - p) ** M for p in _shares(case)), G)
        if fwd:
            n = rows * K + used * N * K + used * N + M * N * (2 if case.get("residual") else 1)
            return {"bytes": b * n, "flops": 2 * M * N * K}
        n = rows * K + used * N * K + M * N * (1 if case["act"] == "none" else 2) + M * K + G * N * (K + 1)
        return {"bytes": b * n, "flops": 4 * M * N * K}
    d, k = case["d"], case["k"]
    n = rows * d * (k + 1 + (1 if case["residual"] else 0))
    if not fwd:
        n += rows * d * (1 + k)
    return {"bytes": b * n + 4 * rows * k * (1 if fwd else 2), "flops": (2 if fwd else 5) * rows * d * k}


# ---- 64 bits, written apart from the plain forms -----------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    return globals()["_exact_" + case["op"]](s, case, D)


def _exact_norm(s, c, D):
    x, w, b = s["X"].to(D), s["weight"].to(D), s["bias"].to(D)
    var, mean = torch.var_mean(x, dim=1, unbiased=False)
    rstd = (var + 1e-5) ** -0.5
    unit = (x - mean[:, None]) * rstd[:, None]
    y = unit * w + b
    if c["dir"] == "fwd":
        return {"Y": y, "mean": mean, "rstd": rstd}
    dy = s["dY"].to(D)
    u = dy * w
    along = (u * unit).sum(1) / c["d"]
    dx = (u - u.sum(1, keepdim=True) / c["d"] - unit * along[:, None]) * rstd[:, None]
    return {"Y": y, "dX": dx, "dweight": (unit * dy).sum(0), "dbias": dy.sum(0)}


def _exact_route(s, c, D):
    """The gradient by differentiating the definition."""
    E, k = c["experts"], c["k"]
    l0 = s["logits"].to(D)
    live = torch.isfinite(l0).any(1)
    if s["valid"] is not None:
        live = live & s["valid"]
    rows = live.nonzero()[:, 0]
    l = l0[rows].clone().requires_grad_(True)
    n = max(1, rows.numel())
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    pick = torch.argsort(l.detach(), dim=1, descending=True, stable=True)[:, :k]
    chosen = l.gather(1, pick)
    has = torch.isfinite(chosen.detach())
    scale = torch.logsumexp(chosen, 1) if c["norm"] == "chosen" else lse
    g = torch.exp(chosen - scale[:, None])
    hits = torch.zeros(E, dtype=D, device=l.device).index_add_(0, pick[has], torch.ones_like(g.detach()[has]))
    f = hits / hits.sum().clamp_min(1)
    losses = torch.stack((E * (f * p.sum(0)).sum() / n, (lse * lse).sum() / n))
    gates = torch.zeros((c["rows"], k), dtype=D, device=l.device)
    gates[rows] = g.detach()
    out = {"ids": None, "gates": gates, "counts": None, "losses": losses.detach()}
    if c["dir"] == "fwd":
        return out
    d = torch.zeros_like(l0)
    if rows.numel():
        weight = torch.where(has, s["d_gates"].to(D)[rows], torch.zeros_like(g.detach()))
        total = (g * weight).sum() + (losses * s["d_losses"].to(D)).sum()
        d[rows] = torch.autograd.grad(total, l)[0].nan_to_num(0.0)
    out["d_logits"] = d
    return out


def _exact_act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def _exact_slope(name, z):
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(_exact_act(name, z).sum(), z)[0]


def _exact_linear(s, c, D):
    x, w = s["X"].to(D), s["W"].to(D)
    if c["dir"] == "fwd":
        y = _exact_act(c["act"], torch.addmm(s["bias"].to(D), x, w.t()))
        return {"Y": y if s["residual"] is None else y + s["residual"].to(D)}
    dz = s["dY"].to(D) * _exact_slope(c["act"], s["pre"].to(D))
    return {"dX": dz @ w, "dW": dz.t() @ x, "dbias": dz.sum(0)}


def _exact_experts(s, c, D):
    """Expert by expert, over the rows that chose it."""
    x, share, fwd = s["X"].to(D), c["share"], c["dir"] == "fwd"
    M = c["rows"] * share
    res = {"Y": x.new_zeros((M, c["n"]))} if fwd else {
        "dX": x.new_zeros((M, c["k_in"])), "dW": x.new_zeros(s["W"].shape), "dbias": x.new_zeros(s["bias"].shape)}
    for e in range(c["experts"]):
        mine = (s["ids"] == e).nonzero()[:, 0]
        w, b = s["W"][e].to(D), s["bias"][e].to(D)
        rows = x[mine // share]
        if fwd:
            res["Y"][mine] = _exact_act(c["act"], rows @ w.t() + b)
        else:
            dz = s["dY"][mine].to(D) * _exact_slope(c["act"], s["pre"][mine].to(D))
            res["dX"][mine] = dz @ w
            res["dW"][e] = dz.t() @ rows
            res["dbias"][e] = dz.sum(0)
    return res


def _exact_combine(s, c, D):
    y, g = s["Y"].to(D), s["gates"].to(D)
    y3 = y.view(c["rows"], c["k"], c["d"])
    out = torch.matmul(g[:, None], y3)[:, 0]
    if s["residual"] is not None:
        out = out + s["residual"].to(D)
    if c["dir"] == "fwd":
        return {"out": out}
    do = s["dOut"].to(D)
    return {"out": out, "dY": torch.repeat_interleave(do, c["k"], 0) * g.reshape(-1, 1),
            "dgates": torch.matmul(y3, do[:, :, None])[:, :, 0]}
