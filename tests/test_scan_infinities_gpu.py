"""The gated recurrence after an infinite value: infinite from there on, however little is left of
a step's factor after many frames, until a document's end; other channels as they were."""
from __future__ import annotations

import math

import pytest
import torch

from tests import test_recurrent_gpu as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300 import ops

    return ops


def passes(ops, x, gate, state, dy, dend, **kw):
    X, G, S = (t.detach().requires_grad_() for t in (x, gate, state))
    y, end = ops.gated_scan(X, G, S, return_state=True, **kw)
    return [y.detach(), end.detach(), *torch.autograd.grad((y, end), (X, G, S), (dy, dend))]


# one block's tile, clusters, and rows cut into stretches; channels on the 16-byte grid and off it
@pytest.mark.parametrize("dtype", base.TYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("T,Cn", [(3, 8), (40, 8), (700, 40), (3000, 129), (26001, 8), (20001, 23)])
def test_infinities_stay(ops, T, Cn, reverse, dtype):
    B = 2
    x, gate, state = (t.contiguous() for t in base.inputs((B, T, Cn), dtype, T, shift=-1.0))
    g = base.gen(3)
    dy, dend = base.randn(g, B, T, Cn, dtype=dtype), base.randn(g, B, Cn)
    clean = passes(ops, x, gate, state, dy, dend, reverse=reverse)
    order = list(range(T))[::-1] if reverse else list(range(T))
    at, back = order[T // 3], order[2 * T // 3]
    x[0, at, 1], x[0, at, 2], dy[1, back, 3] = math.inf, -math.inf, -math.inf
    state[1, 4], dend[1, 5] = math.inf, math.inf
    got = passes(ops, x, gate, state, dy, dend, reverse=reverse)
    walk = (lambda t: t.flip(1)) if reverse else (lambda t: t)
    y, want = walk(got[0]), walk(clean[0])
    n = T // 3
    assert (y[0, n:, 1] == math.inf).all() and (y[0, n:, 2] == -math.inf).all() and (y[1, :, 4] == math.inf).all()
    assert torch.equal(y[0, :n], want[0, :n]) and torch.equal(y[0, :, 3:], want[0, :, 3:])
    assert got[1][0, 1] == math.inf and got[1][0, 2] == -math.inf and got[1][1, 4] == math.inf
    dx, want = walk(got[2]), walk(clean[2])
    n = 2 * T // 3
    assert (dx[1, :n + 1, 3] == -math.inf).all() and (dx[1, :, 5] == math.inf).all()
    assert torch.equal(dx[1, n + 1:, 3], want[1, n + 1:, 3]) and torch.equal(dx[0], want[0])
    assert got[4][1, 3] == -math.inf and got[4][1, 5] == math.inf and torch.equal(got[4][0], clean[4][0])
    # a document's end ends it too
    docs = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    docs[:, T // 2:] = 1
    got, clean = (passes(ops, *(t.nan_to_num(0.0, 0.0, 0.0) if k else t for t in (x, gate, state, dy, dend)), docs=docs,
                         reverse=reverse) for k in (0, 1))
    y, want = got[0], clean[0]
    first, last = (slice(T // 2, T), slice(0, T // 2)) if reverse else (slice(0, T // 2), slice(T // 2, T))
    if T > 3:
        assert torch.equal(y[:, last], want[:, last]) and (y[1, first, 4] == math.inf).all()
        assert torch.equal(got[1], clean[1])
        assert (got[2][1, last, 5] == math.inf).all() and torch.equal(got[2][1, first, 5], clean[2][1, first, 5])
