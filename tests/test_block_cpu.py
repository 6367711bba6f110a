"""The expert-block entry points on the CPU: workspace sizes and refusals, all
of which come before any device call, and the 64-bit references against
automatic differentiation."""
import ctypes
import math
import os

import pytest
import torch

import block_refs as R
import exact_lloyd_means_flashassign_amd as fk

OK, INVALID, UNSUPPORTED, WORKSPACE, NO_DEVICE = range(5)
F32, BF16, F16 = 0, 1, 2
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fk.LIB_PATH):
        from exact_lloyd_means_flashassign_amd import build
        build.build()
    return fk.load()


def said(lib, text):
    return text in lib.fk_last_error().decode()


def test_symbols(lib):
    names = set(fk.declared_symbols())
    assert {"fk_layer_norm", "fk_layer_norm_backward", "fk_layer_norm_backward_workspace_size", "fk_route",
            "fk_route_backward", "fk_route_workspace_size", "fk_linear", "fk_linear_backward",
            "fk_linear_workspace_size", "fk_combine", "fk_combine_backward"} <= names


def test_layer_norm_refusals(lib):
    def norm(dtype=BF16, wdtype=BF16, X=0x10000, ldx=64, rows=4, d=64, w=0x20000, eps=1e-5, Y=0x30000, ldy=64,
             mean=0x40000):
        return lib.fk_layer_norm(dtype, wdtype, P(X), ldx, rows, d, P(w), None, eps, P(Y), ldy, P(mean), None, None)
    assert norm(dtype=3) == INVALID and said(lib, "element type")
    assert norm(wdtype=F16) == UNSUPPORTED
    assert norm(rows=-1) == INVALID and norm(rows=2 ** 31) == INVALID
    assert norm(d=0) == INVALID and norm(d=(1 << 20) + 1) == INVALID
    assert norm(ldx=63) == INVALID and said(lib, "row stride")
    assert norm(X=0) == INVALID and norm(Y=0) == INVALID and said(lib, "Y is NULL")
    assert norm(X=0x10001) == INVALID and said(lib, "aligned")
    assert norm(eps=-1e-9) == INVALID and norm(eps=math.nan) == INVALID and norm(eps=math.inf) == INVALID
    assert norm(Y=0x10002) == INVALID and said(lib, "Y overlaps X")
    assert norm(Y=0x10000, ldy=72) == INVALID            # the same place at another stride
    assert norm(mean=0x30000) == INVALID and said(lib, "mean overlaps Y")

    def back(dY=0x10000, X=0x20000, mean=0x30000, dX=0x40000, dw=0x50000, d=64, ld=64, ws=0x100000, n=1 << 24):
        return lib.fk_layer_norm_backward(BF16, F32, P(dY), ld, P(X), ld, 4, d, P(mean), P(mean), P(0x60000), P(dX), ld,
                                          P(dw), None, P(ws), n, None)
    assert back(mean=0) == INVALID
    assert back(dX=0x20010) == INVALID and said(lib, "dX overlaps X")
    assert back(dw=0x20000) == INVALID and said(lib, "dweight overlaps X")
    assert back(ws=0) == WORKSPACE and back(ws=0x100008) == WORKSPACE and back(n=64) == WORKSPACE
    assert back(dY=0x400000, dX=0x400000, X=0x800000, d=9000, ld=9000) == UNSUPPORTED
    assert lib.fk_layer_norm_backward_workspace_size(-1, 4) == 0
    assert lib.fk_layer_norm_backward_workspace_size(4, 0) == 0
    a, b = (lib.fk_layer_norm_backward_workspace_size(r, 512) for r in (8, 100000))
    assert 0 < a < b <= 64 << 20


def test_route_refusals(lib):
    def route(dtype=F32, l=0x10000, ld=64, T=8, E=64, k=2, norm=0, ids=0x20000, gates=0x30000, counts=0x40000,
              losses=0x50000, ws=0x100000, n=1 << 20):
        return lib.fk_route(dtype, P(l), ld, T, E, k, norm, None, P(ids), P(gates), P(counts), P(losses), P(0x60000),
                            P(ws), n, None)
    assert route(dtype=-1) == INVALID
    assert route(E=0) == INVALID and route(E=1025, ld=2000) == INVALID
    assert route(k=0) == INVALID and route(k=65, E=100, ld=100) == INVALID and route(k=9, E=8) == INVALID
    assert route(T=-1) == INVALID and route(T=2 ** 30, k=2) == INVALID and said(lib, "slots")
    assert route(norm=2) == INVALID and said(lib, "norm")
    assert route(ld=63) == INVALID
    assert route(ids=0) == INVALID and route(counts=0) == INVALID
    assert route(ids=0x20002) == INVALID
    assert route(gates=0x20000) == INVALID and said(lib, "gates overlaps ids")
    assert route(n=8) == WORKSPACE and route(ws=0) == WORKSPACE
    assert lib.fk_route_workspace_size(10, 0) == 0 and lib.fk_route_workspace_size(10, 64) > 0
    st = lib.fk_route_backward(F32, P(0x10000), 64, 8, 64, 2, 0, None, P(0x20000), P(0x30000), P(0x40000), None, None,
                               P(0x10000), None)
    assert st == INVALID and said(lib, "d_logits overlaps logits")


def shape(**kw):
    h = fk._LinearShape()
    for k, v in dict(dict(dtype=BF16, ydtype=BF16, bias_dtype=BF16, act=0, groups=0, share=1, M=64, N=32, K=128,
                          ldx=128, ldw=128, ldr=32, ldy=32, ldpre=32), **kw).items():
        setattr(h, k, v)
    return h


def test_linear_refusals(lib):
    def lin(h, X=0x10000, W=0x20000, b=0x30000, R=0, slots=0, offsets=0, Y=0x40000, pre=0, ws=0x1000000, n=1 << 30):
        return lib.fk_linear(ctypes.byref(h) if h else None, P(X), P(W), P(b), P(R), P(slots), P(offsets), P(Y), P(pre),
                             P(ws), n, None)
    assert lin(None) == INVALID
    for bad in (dict(dtype=5), dict(act=5), dict(act=-1), dict(M=-1), dict(M=2 ** 31), dict(N=0), dict(K=0),
                dict(K=1 << 21), dict(groups=-1), dict(groups=4097), dict(share=0), dict(share=2),
                dict(groups=2, share=3)):
        assert lin(shape(**bad)) == INVALID, bad
        assert lib.fk_linear_workspace_size(ctypes.byref(shape(**bad)), 0) == 0, bad
    assert lin(shape(ydtype=F16)) == UNSUPPORTED and lin(shape(bias_dtype=F16)) == UNSUPPORTED
    assert lin(shape(ldx=127)) == INVALID and lin(shape(ldy=31)) == INVALID
    assert lin(shape(), X=0x10008) == INVALID and said(lib, "16-byte")
    assert lin(shape(), W=0x20002) == INVALID
    assert lin(shape(), slots=0x50000) == INVALID and said(lib, "groups")
    assert lin(shape(groups=2)) == INVALID and said(lib, "offsets")
    assert lin(shape(groups=2, share=2), offsets=0x50000) == INVALID and said(lib, "slot list")
    assert lin(shape(), Y=0x10010) == INVALID and said(lib, "Y overlaps X")
    assert lin(shape(), R=0x40020) == INVALID and said(lib, "residual")   # not the residual's own place
    assert lin(shape(), pre=0x40000) == INVALID and said(lib, "pre overlaps Y")
    assert lin(shape(), ws=0) == WORKSPACE and lin(shape(), n=16) == WORKSPACE

    def back(h, dY=0x10000, X=0x20000, W=0x30000, pre=0x40000, dX=0x50000, dW=0x60000, n=1 << 30):
        return lib.fk_linear_backward(ctypes.byref(h), P(dY), P(X), P(W), P(pre), None, None, P(dX), P(dW), None,
                                      P(0x1000000), n, None)
    assert back(shape(act=2), pre=0) == INVALID and said(lib, "pre is NULL")
    assert back(shape(), dX=0x60000) == INVALID and said(lib, "overlaps")
    assert back(shape(), X=0) == INVALID and back(shape(), W=0) == INVALID
    assert back(shape(), dY=0x10002) == INVALID
    assert back(shape(), n=0) == WORKSPACE


def test_combine_refusals(lib):
    def comb(dtype=BF16, Y=0x10000, rows=4, k=2, d=64, R=0, out=0x20000, ldo=64):
        return lib.fk_combine(dtype, P(Y), rows, k, d, None, P(R), 64, P(out), ldo, None)
    assert comb(dtype=9) == INVALID and comb(k=0) == INVALID and comb(k=65) == INVALID and comb(d=0) == INVALID
    assert comb(Y=0) == INVALID and comb(ldo=60) == INVALID
    assert comb(out=0x10080) == INVALID and said(lib, "out overlaps Y")
    assert comb(rows=2 ** 30, k=4) == INVALID and said(lib, "slots")
    st = lib.fk_combine_backward(BF16, P(0x10000), 64, None, 4, 2, 64, P(0x20000), P(0x30000), P(0x40000), None)
    assert st == INVALID and said(lib, "Y is NULL")


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="a device is visible")
def test_no_device(lib):
    st = lib.fk_combine(BF16, P(0x10000), 4, 2, 64, None, None, 64, P(0x20000), 64, None)
    assert st == NO_DEVICE


def test_binding_rejects_host_tensors(lib):
    X = torch.zeros(8, 16)
    for call in (lambda: fk.fk_layer_norm(X), lambda: fk.fk_route(X, 2), lambda: fk.fk_linear(X, X),
                 lambda: fk.fk_combine(X, 2)):
        with pytest.raises(ValueError):
            call()


# ---- the references themselves ------------------------------------------------


def test_reference_gradients_against_autograd():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, dtype=R.D)  # noqa: E731
    X, w, b, dY = r(5, 12), r(12), r(12), r(5, 12)
    x, w_, b_ = (t.clone().requires_grad_(True) for t in (X, w, b))
    y = torch.nn.functional.layer_norm(x, (12,), w_, b_, 1e-5)
    assert torch.allclose(R.layer_norm(X, w, b, 1e-5)[0], y.detach(), atol=1e-12)
    for a, e in zip(R.layer_norm_grad(dY, X, w, 1e-5)[:3], torch.autograd.grad((y * dY).sum(), (x, w_, b_))):
        assert torch.allclose(a, e, atol=1e-11)

    l, dg, dl = r(9, 7), r(9, 3), torch.tensor([0.4, -0.2], dtype=R.D)
    for norm in ("chosen", "all"):
        ids, gates, _, losses, n, _, _, _, f = R.route(l, 3, norm)
        q = l.clone().requires_grad_(True)
        p = torch.softmax(q, 1)
        pick = q.gather(1, ids.long())
        gt = torch.softmax(pick, 1) if norm == "chosen" else p.gather(1, ids.long())
        ls = torch.stack((7 * (f * p.mean(0)).sum(), torch.logsumexp(q, 1).square().mean()))
        assert torch.allclose(gt, gates) and torch.allclose(ls, losses)
        e = torch.autograd.grad((gt * dg).sum() + (ls * dl).sum(), q)[0]
        assert torch.allclose(R.route_grad(l, 3, norm, None, dg, dl)[0], e, atol=1e-12)

    X, Wt, b, dY = r(4, 6), r(2, 5, 6), r(2, 5), r(8, 5)
    slots = torch.tensor([6, 1, 4, 0, 7, 2, 3, 5], dtype=torch.int32)
    offsets = torch.tensor([0, 3, 7], dtype=torch.int32)  # one slot unrouted
    where = {"slots": slots, "offsets": offsets, "share": 2}
    group = torch.full((8,), 2)
    group[slots[:3].long()], group[slots[3:7].long()] = 0, 1
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        x, w_, b_ = (t.clone().requires_grad_(True) for t in (X, Wt, b))
        z = torch.stack([x[s // 2] @ w_[group[s]].t() + b_[group[s]] if group[s] < 2 else x[0, 0] * torch.zeros(5, dtype=R.D)
                         for s in range(8)])
        fn = {"relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
              "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name]
        y = torch.where((group < 2)[:, None], fn(z), torch.zeros_like(z))
        got, pre, _, _ = R.linear(X, Wt, b, name, None, **where)
        assert torch.allclose(got, y.detach(), atol=1e-12)
        dx, dw, db, *_ = R.linear_grad(dY, X, Wt, name, pre, **where)
        ex, ew, eb = torch.autograd.grad((y * dY).sum(), (x, w_, b_))
        assert torch.allclose(dx.view(4, 2, 6).sum(1), ex, atol=1e-11)
        assert torch.allclose(dw, ew, atol=1e-11) and torch.allclose(db, eb, atol=1e-11)

    Y, gt, do = r(6, 5), r(3, 2), r(3, 5)
    y, q = Y.clone().requires_grad_(True), gt.clone().requires_grad_(True)
    out = (y.view(3, 2, 5) * q[:, :, None]).sum(1)
    assert torch.allclose(R.combine(Y, 2, gt, None)[0], out.detach())
    for a, e in zip(R.combine_grad(do, Y, gt)[:2], torch.autograd.grad((out * do).sum(), (y, q))):
        assert torch.allclose(a, e, atol=1e-12)
