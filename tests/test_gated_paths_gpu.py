"""The recurrent block's operators on the paths that only large, long or lopsided calls take,
against their definitions in 64 bits: sums cut into stretches, more tiles than pairs of SMs,
rows of the recurrence cut into stretches."""
from __future__ import annotations

import pytest
import torch

from tests import recurrent_reference as ref
from tests import test_gated_gpu as gated
from tests import test_recurrent_gpu as base

pytestmark = pytest.mark.gpu

F32, F16, BF16 = gated.F32, gated.F16, gated.BF16


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300 import ops

    return ops


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,K,F", [
    (4100, 72, 136),     # the weights' gradients: few tiles, a long sum
    (200, 130, 1800),    # dx: the same
    (300, 640, 5000),    # the weights' gradients: more tiles than pairs of SMs
    (10300, 520, 72),    # dx: the same
    (5000, 64, 1000),    # both products with pairs of weights: the same
    (20500, 248, 24),    # tiles of all rows and one step of the sum
])
def test_sums_and_tiles(ops, M, K, F, dtype):
    x, wg, wu, dh = gated.make(M, K, F, dtype, M)
    gated.check(ops, x, wg, wu, dh, f"{M} {K} {F}", "gelu")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,F", [(5000, 64, 1000), (130, 512, 12000), (20300, 400, 136)])
def test_tiles_of_8_bits(ops, M, K, F, act, dtype):
    x, wg, wu, _ = gated.make(M, K, F, F32, M)
    x *= torch.linspace(0.1, 30, M, device="cuda")[:, None]
    (x8, sx), (g8, sg), (u8, su) = (ops.rows_8bit(t) for t in (x, wg, wu))
    h = ops.gated_linear_8bit(x8, sx, g8, sg, u8, su, act, dtype)
    want = ref.gated(x8.float(), g8.float(), u8.float(), act, scales=(sx, sg, su), dtype=dtype, unit=2 * ref.E)
    ref.close(h, *want["out"], act)


def walk(f, b, first):
    """h_t = f_t h_(t-1) + b_t along dim 1 from `first`: h after each frame, and before it."""
    B, T, C = b.shape
    L = max(1, int(T ** 0.5))
    n = -(-T // L)
    f = torch.nn.functional.pad(f, (0, 0, 0, n * L - T), value=1.0).reshape(B, n, L, C)
    h = torch.nn.functional.pad(b, (0, 0, 0, n * L - T)).reshape(B, n, L, C).clone()
    reach = f.clone()
    for t in range(1, L):
        h[:, :, t] += f[:, :, t] * h[:, :, t - 1]
        reach[:, :, t] *= reach[:, :, t - 1]
    state = first
    for k in range(n):
        h[:, k] += reach[:, k] * state[:, None]
        state = h[:, k, -1]
    h = h.reshape(B, n * L, C)[:, :T]
    return h, torch.cat([first[:, None], h[:, :-1]], 1)


def long_scan(x, gate, state, lens, docs, reverse, dy, dend):
    """ref.scan, its bounds included, by pieces of the row side by side."""
    E, u, tiny = ref.E, ref.U[x.dtype], ref.TINY[x.dtype]
    B, T, C = x.shape
    turn = (lambda t: t.flip(1)) if reverse else (lambda t: t)
    used, new = (torch.full((B, T), v, dtype=torch.bool, device="cuda") for v in (True, False))
    if lens is not None:
        used &= turn(torch.arange(T, device="cuda")[None, :] < lens[:, None])
    if docs is not None:
        ids = turn(docs)
        used &= ids >= 0
        new[:, 1:] = ids[:, 1:] != ids[:, :-1]
    used, new = used[:, :, None], (new & used)[:, :, None]
    xs, gs = (torch.where(used, turn(t).double(), 0.0) for t in (x, gate))
    a, rest = torch.sigmoid(gs), torch.sigmoid(-gs)
    ra, rr = a * (rest * (gs.abs() + 8) * E + 4 * E), rest * (gs.abs() + 12) * E
    f = torch.where(new, 0.0, torch.where(used, a, 1.0))
    first = state.double()
    on = lambda v: torch.where(used, v, 0.0)  # noqa: E731
    go = lambda v: torch.where(used & ~new, v, 0.0)  # noqa: E731
    h, h0 = walk(f, on(rest * xs), first)
    m, m0 = walk(f, on(rest * xs.abs()), first.abs())
    h0, m0 = go(h0), go(m0)
    e, e0 = walk(f, on(m0 * (ra + 6 * E * a) + xs.abs() * (rr + 6 * E * rest)), torch.zeros_like(first))
    e0 = go(e0)
    got = {"out": (turn(on(h)), turn(on(u * h.abs() + e + 64 * E * m + tiny))),
           "state": (h[:, -1], e[:, -1] + 64 * E * m[:, -1] + 1e-30)}
    back = lambda v: v.flip(1)  # noqa: E731
    g, d, nothing = on(turn(dy).double()), dend.double(), torch.zeros_like(first)
    after, d0 = walk(back(f), back(go(a * g)), d)
    sizes, s0 = walk(back(f), back(go(a * g.abs())), d.abs())
    dh, dm = g + back(d0), g.abs() + back(s0)
    off, o0 = walk(back(f), back(go(dm * (ra + 8 * E * a))), nothing)
    de = back(o0) + 64 * E * dm
    far = h0 - xs
    got["dx"] = (turn(on(rest * dh)), turn(on((u + 4 * E) * (rest * dh).abs() + rest * de + rr * dm + tiny)))
    dg = dh * far * a * rest
    got["dgate"] = (turn(on(dg)), turn(on(
        (u + 8 * E) * dg.abs() + tiny + a * rest * (de * far.abs() + dm * (e0 + 64 * E * m0 + 2 * E * far.abs()))
        + dm * far.abs() * (a * rr + rest * ra))))
    got["dstate"] = (after[:, -1], off[:, -1] + 64 * E * sizes[:, -1] + 1e-30)
    return got


def agree(a, b):
    for name in a:
        for u, v in zip(a[name], b[name]):
            assert (u - v).abs().max() <= 1e-9 * (1 + v.abs().max()), name


@pytest.mark.parametrize("dtype", gated.TYPES)
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("T,C", [(150, 3), (26001, 5), (26001, 16), (100003, 8)])
def test_stretches_frame_by_frame(ops, T, C, reverse, dtype):
    # every frame within its own bound, some roundings of what it remembers
    B = 2
    x, gate, state = base.inputs((B, T, C), dtype, 12)
    g = base.gen(3)
    dy, dend = base.randn(g, B, T, C, dtype=dtype), base.randn(g, B, C)
    docs = (torch.arange(T, device="cuda", dtype=torch.int32) // (T // 5)).repeat(B, 1)
    docs[1, T // 2:T // 2 + 30] = -1
    docs[0, T // 3] = 77  # a document of one frame
    for kw in ({}, {"docs": docs, "lens": torch.tensor([T, T - T // 9], dtype=torch.int32, device="cuda")}):
        want = long_scan(x, gate, state, kw.get("lens"), kw.get("docs"), reverse, dy, dend)
        if T < 1000:
            agree(want, ref.scan(x, gate, state, dy=dy, dend=dend, reverse=reverse, **kw))
        X, G, S = (t.detach().requires_grad_() for t in (x, gate, state))
        out = ops.gated_scan(X, G, S, return_state=True, reverse=reverse, **kw)
        ref.close(out[0], *want["out"], f"{list(kw)}: out")
        ref.close(out[1], *want["state"], f"{list(kw)}: state")
        for name, t in zip(("dx", "dgate", "dstate"), torch.autograd.grad(out, (X, G, S), (dy, dend))):
            ref.close(t, *want[name], f"{list(kw)}: {name}")
