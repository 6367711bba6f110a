"""The activations and their slopes in fp32 against 64 bits, value by value: a
sum of one product (1 times z) leaves the activation alone.

Bounds, in units of w = 2^-24 (the relative error of one rounding).  The
library's exponential and complementary error function are within 2 and 4 ulp,
4 w and 8 w; a sum, product or quotient adds 1 w; an exponential whose argument
is off by e is off by e relative, a function f whose argument is off by e
relative by e |x f'(x) / f(x)|.
"""
import math

import pytest
import torch

import block_refs as R
from block_refs import check
from gpu_helpers import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = R.D


def cdf_rel(z):
    """Relative bound of erfc(-z / sqrt 2) / 2: the argument takes two roundings
    (the constant's and the product's)."""
    t = -z / math.sqrt(2)
    c = torch.special.erfc(t)
    bend = torch.where(c > 0, 2 * t.abs() * torch.exp(-t * t) / (math.sqrt(math.pi) * c), torch.zeros_like(t))
    return 8 + 2 * bend


def logistic_rel(x, arg):
    """Relative bound of 1 / (1 + e^-x) with x off by `arg` relative."""
    return 6 + (4 + arg * x.abs()) * torch.sigmoid(-x)


def tanh_arg(z):
    return 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


TANH_ARG = 7  # two constants, three products of the cube, a sum, a product


def value(name, z):
    """act(z) and its bound."""
    y = R.act(name, z)
    if name == "gelu":
        rel = cdf_rel(z) + 1
    elif name == "gelu_tanh":
        rel = logistic_rel(tanh_arg(z), TANH_ARG) + 1
    else:
        rel = logistic_rel(z, 0) + 1
    return y, rel * R.W * y.abs()


def slope(name, z):
    """act'(z) and its bound."""
    s = R.act_slope(name, z)
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        t = z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        # the exponent z^2 / 2 takes two roundings; constant, two products and the sum
        e = cdf_rel(z) * c + (4 + z * z + 3) * t.abs() + s.abs()
    else:
        x = z if name == "silu" else tanh_arg(z)
        arg = 0 if name == "silu" else TANH_ARG
        p = torch.sigmoid(x)
        q = torch.sigmoid(-x)
        e_p = logistic_rel(x, arg) * p      # and of 1 - p, with a rounding of its own
        f = z if name == "silu" else z * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        # p + p q f: f takes up to 7 roundings, the products and sums 5
        e = e_p * (1 + q * f).abs() + p * f.abs() * (e_p + q) + 12 * p * q * f.abs() + 2 * p + s.abs()
    return s, e * R.W


def inputs(lo, dtype):
    """Values from lo to 12 that dtype holds, dense around 0, and tiny ones."""
    z = torch.cat((torch.linspace(lo, 12, 4001), torch.linspace(-3, 3, 2001),
                   torch.tensor([0.0, 1e-6, -1e-6, 2.0 ** -20, -2.0 ** -20])))
    return z.to(dtype)


@pytest.mark.parametrize("rows", [1, 40])  # a few rows, and tiles
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name,lo", [("gelu", -12.0), ("gelu_tanh", -8.0), ("silu", -60.0)])
def test_activation_in_fp32(gpu_lib, name, lo, dtype, rows):
    """An fp32 result is as good from 16-bit operands as from fp32 ones."""
    fk = gpu_lib
    log(f"{name} {dtype} rows={rows}")
    z = inputs(lo, dtype)
    X = torch.ones((rows, 1), dtype=dtype, device=DEV)
    Y, _ = fk.fk_linear(X, z.to(DEV)[:, None].contiguous(), act=name, out_dtype=torch.float32)
    y, e = value(name, z.to(D))
    for r in {0, rows - 1}:
        check(f"{name} row {r}", Y[r], y, e, torch.float32)


@pytest.mark.parametrize("name,lo", [("gelu", -12.0), ("gelu_tanh", -8.0), ("silu", -60.0)])
def test_slope_in_fp32(gpu_lib, name, lo):
    """db of one row of ones is the slope itself."""
    fk = gpu_lib
    log(f"slope of {name}")
    z = inputs(lo, torch.float32).to(DEV)
    X = torch.ones((1, 1), device=DEV)
    _, dW, db = fk.fk_linear_backward(torch.ones((1, z.numel()), device=DEV), X, z[:, None].contiguous(), act=name,
                                      pre=z[None].contiguous())
    s, e = slope(name, z.cpu().to(D))
    check(f"slope of {name}", db, s, e, torch.float32)
    assert torch.equal(dW[:, 0], db)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_activations_far_out(gpu_lib, dtype):
    """Past the range of the exponential: z, 0 or NaN as the formulas have it."""
    fk = gpu_lib
    inf, nan = math.inf, math.nan
    z = torch.tensor([-1e30, -300.0, -100.0, 100.0, 300.0, 1e30, inf, nan], dtype=dtype, device=DEV)
    X = torch.ones((1, 1), dtype=dtype, device=DEV)
    for name in ("gelu", "gelu_tanh", "silu"):
        Y = fk.fk_linear(X, z[:, None].contiguous(), act=name, out_dtype=torch.float32)[0][0].cpu()
        assert torch.equal(Y[3:7], z[3:7].float().cpu()) and torch.isnan(Y[7]), (name, Y)
        assert (Y[:3].abs() < 1e-30).all(), (name, Y)
        one = torch.ones((1, 7), dtype=dtype, device=DEV)
        db = fk.fk_linear_backward(one, X, z[:7, None].contiguous(), act=name, pre=z[None, :7].contiguous(),
                                   with_dx=False)[2].float().cpu()
        assert torch.equal(db[3:], torch.ones(4)) and (db[:3].abs() < 1e-30).all(), (name, db)
