"""A routed expert block, trained and then used row by row.

    x -> layer norm -> router -> top-k experts (up, silu, down) -> weighted sum + x

The router's rows start as the spherical k-means centroids of the normalised
inputs (fk_fit), so every expert begins with one cluster of the data; training
then moves router and experts together, with the balance loss holding the loads
even.  The data is synthetic: a mixture of clusters, each with a linear map of
its own that its expert has to learn.

    python examples/expert_block.py [--steps 60] [--rows 8192] [--dim 256] [--experts 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import exact_lloyd_means_flashassign_amd as fk  # noqa: E402


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = fk.fk_layer_norm(x, weight, bias)
        ctx.save_for_backward(x, mean, rstd, weight)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        return fk.fk_layer_norm_backward(dy.contiguous(), x, mean, rstd, weight)


class Linear(torch.autograd.Function):
    """fk_linear; `where` holds the slots, offsets and share of a grouped one."""

    @staticmethod
    def forward(ctx, x, weight, bias, act, where, out_dtype):
        y, pre = fk.fk_linear(x, weight, bias, act=act, with_pre=act != "none", out_dtype=out_dtype, **where)
        ctx.save_for_backward(x, weight, pre)
        ctx.rest = (act, where, None if bias is None else bias.dtype)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, pre = ctx.saved_tensors
        act, where, bias_dtype = ctx.rest
        dx, dw, db = fk.fk_linear_backward(dy.contiguous(), x, weight, act=act, pre=pre,
                                           with_bias=bias_dtype is not None, bias_dtype=bias_dtype, **where)
        if where.get("share", 1) > 1:
            dx = fk.fk_combine(dx, where["share"])  # the slots of a row add up
        return dx, dw, db, None, None, None


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        ids, gates, counts, losses, live = fk.fk_route(logits, k)
        ctx.save_for_backward(logits, ids, counts, live)
        ctx.mark_non_differentiable(ids, counts)
        return ids, gates, counts, losses

    @staticmethod
    def backward(ctx, _ids, d_gates, _counts, d_losses):
        logits, ids, counts, live = ctx.saved_tensors
        return fk.fk_route_backward(logits, ids, counts, live, d_gates.contiguous(), d_losses.contiguous()), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, gates, residual):
        ctx.save_for_backward(y, gates)
        return fk.fk_combine(y, gates.shape[1], gates, residual=residual)

    @staticmethod
    def backward(ctx, d_out):
        y, gates = ctx.saved_tensors
        d_out = d_out.contiguous()
        dy, dgates = fk.fk_combine_backward(d_out, y, gates)
        return dy, dgates, d_out


class ExpertBlock(torch.nn.Module):
    def __init__(self, dim, hidden, experts, k, dtype=torch.bfloat16, device="cuda"):
        super().__init__()

        def normal(*shape, scale):
            return torch.nn.Parameter(torch.randn(shape, device=device) * scale)
        self.k, self.dtype = k, dtype
        self.norm_weight = torch.nn.Parameter(torch.ones(dim, device=device))
        self.norm_bias = torch.nn.Parameter(torch.zeros(dim, device=device))
        self.router = normal(experts, dim, scale=dim ** -0.5)
        self.up = normal(experts, hidden, dim, scale=dim ** -0.5)
        self.up_bias = torch.nn.Parameter(torch.zeros(experts, hidden, device=device))
        self.down = normal(experts, dim, hidden, scale=0.1 * hidden ** -0.5)

    @torch.no_grad()
    def route_by_clusters(self, x, iterations=10, sharpness=4.0):
        """The router's rows become the spherical centroids of the normalised rows."""
        h, _, _ = fk.fk_layer_norm(x.float(), self.norm_weight, self.norm_bias)
        centroids, _, counts = fk.fk_fit(h, K=self.router.shape[0], n_iter=iterations, metric="spherical")
        self.router.copy_(centroids * sharpness / x.shape[1] ** 0.5)
        return counts

    def forward(self, x):
        d, experts = self.dtype, self.router.shape[0]
        h = LayerNorm.apply(x, self.norm_weight.to(d), self.norm_bias.to(d))
        logits = Linear.apply(h, self.router.to(d), None, "none", {}, torch.float32)
        ids, gates, counts, losses = Route.apply(logits, self.k)
        slots, offsets = fk.fk_sort_inverse(ids.view(-1), experts + 1)
        where = {"slots": slots, "offsets": offsets}
        a = Linear.apply(h, self.up.to(d), self.up_bias, "silu", {**where, "share": self.k}, None)
        y = Linear.apply(a, self.down.to(d), None, "none", where, None)
        return Combine.apply(y, gates, x), losses, counts


def mixture(rows, dim, clusters, seed, device="cuda"):
    """Rows from a mixture of clusters, and what the block should make of them."""
    g = torch.Generator(device=device).manual_seed(seed)
    centers = torch.randn((clusters, dim), generator=g, device=device) * 2
    maps = torch.randn((clusters, dim, dim), generator=g, device=device) * dim ** -0.5
    which = torch.randint(0, clusters, (rows,), generator=g, device=device)
    x = (centers[which] + torch.randn((rows, dim), generator=g, device=device)).bfloat16()
    target = torch.empty((rows, dim), device=device)
    for c in range(clusters):
        mine = which == c
        target[mine] = x[mine].float() + x[mine].float() @ maps[c]
    return x, target


def train(steps=60, rows=8192, dim=256, experts=16, k=2, seed=0, log=print):
    torch.manual_seed(seed)
    x, target = mixture(rows, dim, experts, seed)
    block = ExpertBlock(dim, 2 * dim, experts, k)
    counts = block.route_by_clusters(x)
    log(f"clusters: {int(counts.min())} to {int(counts.max())} of {rows} rows")
    opt = torch.optim.AdamW(block.parameters(), lr=3e-3, weight_decay=0.0)
    history = []
    for step in range(steps):
        opt.zero_grad(set_to_none=True)
        out, losses, counts = block(x)
        error = (out.float() - target).square().mean()
        (error + 0.01 * losses[0] + 1e-4 * losses[1]).backward()
        opt.step()
        history.append(error.detach())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step}: error {float(history[-1]):.4f}, balance {float(losses[0].detach()):.3f}, loads "
                f"{int(counts.min())} to {int(counts.max())}")
    return block, x, torch.stack(history)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 60), ("rows", 8192), ("dim", 256), ("experts", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block, x, _ = train(a.steps, a.rows, a.dim, a.experts)
    with torch.no_grad():  # a row at a time, as a decoding step would
        whole = block(x[:4])[0]
        alone = torch.cat([block(x[i:i + 1])[0] for i in range(4)])
    print(f"four rows one by one differ from the same four together by {float((whole - alone).abs().max()):.3g}")
