"""Gradients of the gated linear layer in f16 where its projections, or its rows, are far from
one another in size: bounds relative to the terms that each result is the sum of."""
from __future__ import annotations

import pytest
import torch

from tests import recurrent_reference as ref
from tests.test_gated_gpu import gen, randn

pytestmark = pytest.mark.gpu

F16 = torch.float16
U, TINY, E = ref.U[F16], ref.TINY[F16], ref.E


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300 import ops

    return ops


def check(ops, x, wg, wu, dh, kind, what):
    """dx and the weights' gradients: dg and du are rounded to f16 relative to themselves whatever
    their size, results once more; sums are off by 2 E a term, the activation's slope by the
    error that this gives g and by its own few roundings (128 E of the terms it is made of)."""
    leaves = [t.detach().requires_grad_() for t in (x, wg, wu)]
    got = torch.autograd.grad(ops.gated_linear(*leaves, kind), leaves, dh)
    X, G, P, D = (t.double() for t in (x, wg, wu, dh))
    g, p = X @ G.T, X @ P.T
    K = x.shape[1]
    eg, ep = (2 * (K + 16) * E * (X.abs() @ W.abs().T) for W in (G, P))
    a, slope, most, bend = ref.act(g, kind)
    dg, du = D * p * slope, D * a
    # a and its slope are no larger than the terms 1 and |g| in any of them
    es = bend * eg + 128 * E * (1 + g.abs())
    ea = most * eg + 128 * E * g.abs().clamp(min=float(kind == "sigmoid"))
    ed = U * dg.abs() + D.abs() * (p.abs() * es + slope.abs() * ep + es * ep)
    eu = U * du.abs() + D.abs() * ea
    sums = lambda n: 2 * (n + 16) * E  # noqa: E731
    F, M = wg.shape[0], x.shape[0]
    want = dg @ G + du @ P
    size = dg.abs() @ G.abs() + du.abs() @ P.abs()
    ref.close(got[0], want, U * want.abs() + ed @ G.abs() + eu @ P.abs() + sums(2 * F) * size + TINY, what + ": dx")
    for name, t, d, e in (("dw_gate", got[1], dg, ed), ("dw_up", got[2], du, eu)):
        want = d.T @ X
        ref.close(t, want, U * want.abs() + e.T @ X.abs() + sums(M) * (d.abs().T @ X.abs()) + TINY, f"{what}: {name}")


@pytest.mark.parametrize("kind", ["silu", "gelu", "sigmoid", "relu"])
@pytest.mark.parametrize("M,K,F", [(40, 64, 72), (300, 63, 130)])
def test_projections_of_any_size(ops, M, K, F, kind):
    g = gen(M)
    x, wg, dh = randn(g, M, K, dtype=F16), randn(g, F, K, scale=K ** -0.5), randn(g, M, F)
    unit = randn(g, F, K, scale=K ** -0.5)
    # what w_up gives is beyond what f16 holds, dh and w_gate are small enough for all results
    check(ops, x, (wg * 2 ** -6).to(F16), (unit * 3e4).to(F16), (dh * 2 ** -10).to(F16), kind, "loud up")
    check(ops, x, (wg * 2 ** -2).to(F16), (unit * 2 ** -12).to(F16), dh.to(F16), kind, "quiet up")
    check(ops, (x * 2 ** -4), (wg * 2 ** -6).to(F16), (unit * 2 ** -6).to(F16), dh.to(F16), kind, "quiet all")
    check(ops, x, wg.to(F16), unit.to(F16), (dh * 2 ** -14).to(F16), kind, "quiet gradients")
    check(ops, x * 2 ** 8, (wg * 2 ** -8).to(F16), (unit * 2 ** -8).to(F16), (dh * 2 ** -6).to(F16), kind, "loud rows")


def test_a_quiet_projection_of_many_rows(ops):
    # dg of about 2^-21 each, of which the weights' gradient sums 4096 of one sign
    M, F, g = 4096, 40, gen(1)
    x, wg, wu = torch.zeros(M, 16), torch.zeros(F, 16), torch.zeros(F, 16)
    r = lambda *s: torch.rand(*s, generator=torch.Generator().manual_seed(2)) + 1  # noqa: E731
    x[:, 0], x[:, 1] = 1, r(M) * 2 ** -8
    wg[:, 0], wu[:, 1] = r(F) - 1.5, r(F) * 2 ** -13
    dh = r(M, F) / 2
    x, wg, wu, dh = (t.cuda().to(F16) for t in (x, wg, wu, dh))
    for kind in ("silu", "sigmoid"):
        check(ops, x, wg, wu, dh, kind, kind)


def test_gradients_that_are_nothing(ops):
    # rows without a gradient, without inputs, weights of nothing: zeros, and the others as they are
    g = gen(4)
    x, wg, wu, dh = (randn(g, *s, dtype=F16, scale=0.3) for s in ((50, 40), (24, 40), (24, 40), (50, 24)))
    dh[3:20], x[10:30] = 0, 0
    x[5] *= 2 ** 12
    for kind in ("silu", "sigmoid"):
        check(ops, x, wg, wu, dh, kind, "rows")
        check(ops, x, wg, wu * 0, dh, kind, "no up")
        check(ops, x, wg * 0, wu, dh, kind, "no gate")
        check(ops, x, wg, wu, dh * 0, kind, "no gradient")
        check(ops, x * 0, wg, wu, dh, kind, "no input")


@pytest.mark.parametrize("far", [2.0 ** 8, 2.0 ** 16, 2.0 ** 22])
def test_what_only_quiet_rows_hold(ops, far):
    # columns of x that are 0 in the rows with the large gradients: their sums keep their digits
    M, K, F, g = 200, 72, 64, gen(7)
    x, wg, wu = randn(g, M, K, dtype=F16), randn(g, F, K, dtype=F16, scale=0.1), randn(g, F, K, dtype=F16, scale=0.1)
    dh = randn(g, M, F)
    quiet = torch.arange(M, device="cuda") % 4 != 0
    dh = (torch.where(quiet[:, None], dh, dh * far) * 2.0 ** -11).to(F16)
    x[:, ::3] *= torch.where(quiet, 0.05, 0.0).to(F16)[:, None]
    x[:, 1::3] *= torch.where(quiet, 0.0, 1.0).to(F16)[:, None]
    for kind in ("silu", "sigmoid"):
        check(ops, x, wg, wu, dh, kind, kind)
    # sizes of x that undo those of the gradients, and ones that add to them
    size = torch.where(quiet, 1.0, far ** -0.5).to(F16)[:, None]
    check(ops, x * size, wg, wu, dh, "silu", "undone")
    check(ops, x * size.flip(0), wg, wu, dh, "silu", "other rows")


def test_loud_rows_change_no_bit_of_others_dx(ops):
    M, K, F, g = 150, 72, 130, gen(8)
    x, wg, wu = randn(g, M, K, dtype=F16), randn(g, F, K, dtype=F16, scale=0.1), randn(g, F, K, dtype=F16, scale=0.1)
    dh = randn(g, M, F, dtype=F16, scale=2.0 ** -11)
    dh[5] *= torch.logspace(0, -4, F, device="cuda").to(F16)
    rest = torch.arange(M, device="cuda") != 3
    got = []
    for loud in (1.0, 2.0 ** 13, 2.0 ** 24):
        a, d = x.clone(), dh.clone()
        a[3] *= min(loud, 2.0 ** 8)
        d[3] = (d[3].float() * min(loud, 2.0 ** 22)).to(F16)
        leaves = [t.requires_grad_() for t in (a, wg.clone(), wu.clone())]
        got.append(torch.autograd.grad(ops.gated_linear(*leaves), leaves, d)[0][rest])
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("K", [64, 1 << 21])
def test_projections_that_reach_their_bound(ops, K):
    # x and w_up along one line, so that u is the product of their norms; the largest gradients
    # and slopes of a row beside it
    M, F, g = 40, 8, gen(9)
    line = torch.where(torch.rand(K, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    x = (line * torch.exp2(-6 - torch.arange(M, device="cuda") % 3)[:, None]).to(F16)
    wu = (line * 2.0 ** -4).expand(F, K).to(F16)
    wg = (line * 2.0 ** 7 / K).expand(F, K).to(F16)
    dh = torch.full((M, F), 1.998, device="cuda", dtype=F16)
    dh[:, 1::2] = -1.0
    for kind in ("silu", "gelu", "relu", "sigmoid"):
        check(ops, x, wg, wu, dh, kind, kind)
