"""The gated linear layer where its activation, or what it is multiplied with, is far from
one: bounds relative to what comes out, not to the largest that could."""
from __future__ import annotations

import math

import pytest
import torch

from tests import recurrent_reference as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
E = ref.E
# f32: the FP32 pipes; 16 bits: up to 32 rows by the few rows' kernel, above by the matrix unit's
ROWS = [1, 20, 40]


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300 import ops

    return ops


def one_unit_each(g, u, rows, dtype):
    """x and weights of width 8 whose projections are g and u themselves, one value a unit."""
    x = torch.zeros(rows, 8, device="cuda", dtype=dtype)
    x[:, 0] = 1
    wg, wu = (torch.zeros(len(g), 8, device="cuda", dtype=dtype) for _ in range(2))
    wg[:, 0], wu[:, 0] = g.to(dtype), u.to(dtype)
    return x, wg, wu


def largest_of(dtype):
    return {F32: 2.0 ** 100, F16: 2.0 ** 14, BF16: 2.0 ** 100}[dtype]


def lift(v, dtype):
    """Powers of two that bring the magnitudes v to about one, as far as the type has them."""
    return torch.exp2(-torch.log2(v.abs()).round()).clamp(max=largest_of(dtype))


def act(g, kind):
    """The activation, its slope, and the magnitude of the slope's terms."""
    if kind == "gelu":
        c, pdf = 0.5 * torch.erfc(-g * math.sqrt(0.5)), torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return g * c, c + g * pdf, c + (g * pdf).abs()
    p, q = torch.sigmoid(g), torch.sigmoid(-g)
    if kind == "sigmoid":
        return p, p * q, p * q
    return g * p, p + g * p * q, p + (g * p * q).abs()


def check_act(ops, kind, g, rows, dtype, rel, train=True):
    """act(g) u and, by dh of one row, dg and du themselves; rel(g): the relative error in 32 bits."""
    g = g.to(dtype).double()
    a, slope, terms = act(g, kind)
    unit, tiny = ref.U[dtype], ref.TINY[dtype]
    u = lift(a, dtype)
    x, wg, wu = one_unit_each(g, u, rows, dtype)
    h = ops.gated_linear(x, wg, wu, kind)
    want = a * u
    ref.close(h, want.expand(rows, -1), ((unit + rel(g)) * want.abs() + tiny).expand(rows, -1), f"{kind}: h")
    if not train:
        return
    # dw_gate's first column is dg of that row, dw_up's is du
    u = lift(slope, dtype)
    x, wg, wu = one_unit_each(g, u, rows, dtype)
    leaves = [t.requires_grad_() for t in (x, wg, wu)]
    dh = torch.zeros(rows, len(g), device="cuda", dtype=dtype)
    dh[0] = 1
    dg, du = (t[:, 0] for t in torch.autograd.grad(ops.gated_linear(*leaves, kind), leaves[1:], dh))
    # rounded to the type before the product and after it
    ref.close(dg, u * slope, 2 * unit * (u * slope).abs() + rel(g) * u * terms + 2 * tiny, f"{kind}: dg")
    ref.close(du, a, (2 * unit + rel(g)) * a.abs() + 2 * tiny, f"{kind}: du")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", ROWS)
def test_gelu_of_what_is_far_below_zero(ops, rows, dtype):
    # erfc's relative slope is x^2 2 + 1 = g^2 + 1 times its argument's two roundings, its own
    # error 4 of its last places; on the matrix unit's side exp(-g^2 / 2) with three
    # roundings of its exponent, a polynomial and two approximate instructions
    g = -torch.linspace(0.25, 8, 256, device="cuda")
    check_act(ops, "gelu", g, rows, dtype, lambda g: (2 * g * g + 32) * E)
    check_act(ops, "gelu", -g, rows, dtype, lambda g: 32 * E)


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
def test_exponentials_in_32_bits(ops, kind, rows):
    # exp is off by two of its last places, then a sum, a division and two products
    g = torch.linspace(-80, 80, 321, device="cuda")
    check_act(ops, kind, g, rows, F32, lambda g: 16 * E)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", ROWS)
def test_slopes_of_saturated_sigmoids(ops, rows, dtype):
    # the exponent g log2(e) with two roundings, two approximate instructions, two products
    g = torch.linspace(-11 if dtype is F16 else -40, 11 if dtype is F16 else 40, 161, device="cuda")
    check_act(ops, "sigmoid", g, rows, dtype, lambda g: (2 * g.abs() + 24) * E)
    check_act(ops, "silu", g, rows, dtype, lambda g: (2 * g.abs() + 24) * E)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 20, 40])
def test_scales_far_apart(ops, rows, dtype):
    # scales of rows and of weights whose product passes the range of floats at either end
    # while the projections do not: a sum that is 0 stays 0, a small one keeps its digits
    K, F = 32, 24
    eight = torch.float8_e4m3fn
    x, wg, wu = torch.zeros(rows, K, device="cuda"), torch.zeros(F, K, device="cuda"), torch.zeros(F, K, device="cuda")
    x[:, ::2], wg[1, 1::2], wu[1] = 448, 448, 1    # unit 1: a sum of nothing but zeros
    wg[2], wu[2] = 448, 448
    sx, sg, su = (torch.ones(n, device="cuda") for n in (rows, F, F))
    sx[0], sg[1], su[1] = 1e30, 1e10, 1e-30        # 1e40 times 0
    sx[1], sg[2], su[2] = 1e-10, 1e-30, 1e37       # 1e-40 times 3e6: g = 3.2e-34, u = 3.2e33
    h = ops.gated_linear_8bit(x.to(eight), sx, wg.to(eight), sg, wu.to(eight), su, "silu", dtype)
    assert (h[0, 1] == 0).all()
    total = 448.0 * 448.0 * (K // 2)
    g, u = (total * float(sx[1].double()) * float(s[2].double()) for s in (sg, su))
    want = torch.tensor(g / 2 * u, dtype=torch.float64)
    # four products, the sum (exact), the activation's few roundings, one to the type
    ref.close(h[1, 2], want, (24 * E + ref.U[dtype]) * want, "far apart")
