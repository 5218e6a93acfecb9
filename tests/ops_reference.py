"""The frame-encoder operators in 64 bits from their definitions, with bounds on
the rounding errors of a computation that holds sums in 32 bits and rounds
inputs of its products and its results to the tensors' type once each.

u is the unit roundoff of the tensors' type, e = 2^-24 that of the sums. A
product of n terms summed in any order in 32 bits is off by at most n e times
the sum of its terms' magnitudes.
"""
from __future__ import annotations

import math

import torch

E = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-30, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-30}  # half a subnormal step, rounded up


def bucket(offset: int, num_buckets: int, max_distance: int, bidirectional: bool) -> int:
    """In whole numbers, straight from fm_ops.h."""
    side = num_buckets // 2 if bidirectional else num_buckets
    e, n = side // 2, abs(offset) if bidirectional else max(-offset, 0)
    L = side - e
    c = n
    if n >= e:
        m = max((m for m in range(L) if n ** L >= e ** (L - m) * max_distance ** m), default=0)
        c = e + m
    return c + (side if bidirectional and offset > 0 else 0)


def bucket_tensor(low: int, high: int, *config) -> torch.Tensor:
    D = config[1]
    known = {o: bucket(o, *config) for o in range(-D, D + 1)}
    return torch.tensor([known[max(-D, min(D, o))] for o in range(low, high + 1)], dtype=torch.long)


def close(got: torch.Tensor, want: torch.Tensor, bound: torch.Tensor, what: str) -> None:
    got = got.detach().double().cpu()
    want, bound = want.cpu(), bound.cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= bound)
    bad &= ~(torch.isnan(got) & torch.isnan(want)) & ~(got == want)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        ratio = ((got - want).abs() / bound).nan_to_num(nan=math.inf).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at {at}: "
                             f"{got[at]} against {want[at]} +- {bound[at]}; worst ratio {float(ratio):.3g}")


# ---------------------------------------------------------------------------

def norm(x, weight, bias, eps, dy=None):
    """{name: (value, bound)} of layer norm and, with dy, its gradients."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    up = U[weight.dtype] if weight is not None else u
    tp = TINY[weight.dtype] if weight is not None else tiny
    N = x.shape[-1]
    lead = x.shape[:-1]
    x = x.double().reshape(-1, N)
    w = torch.ones(N, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros(N, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    sd = ((c * c).mean(-1, keepdim=True) + eps).sqrt()
    n = c / sd
    out = n * w + b
    # the mean is off by N e mean|x| at most, every deviation by that and its
    # own rounding; the deviations' squares add N e relative to rstd
    dev = (N + 2) * E * x.abs().mean(-1, keepdim=True) + E * c.abs()
    rel = (N + 8) * E + dev.mean(-1, keepdim=True) / sd
    nb = dev / sd + n.abs() * rel
    got = {"out": (out.reshape(*lead, N), (u * out.abs() + nb * w.abs() + 4 * E * (n * w).abs() + tiny).reshape(*lead, N))}
    if dy is None:
        return got
    dy = dy.double().reshape(-1, N)
    h = dy * w
    mh, mhn = h.mean(-1, keepdim=True), (h * n).mean(-1, keepdim=True)
    dx = (h - mh - n * mhn) / sd
    ah, ahn = h.abs().mean(-1, keepdim=True), (h * n).abs().mean(-1, keepdim=True)
    bound = (N + 8) * E * (h.abs() + ah + n.abs() * ahn) + nb * ahn + n.abs() * (h.abs() * nb).mean(-1, keepdim=True)
    dxb = u * dx.abs() + (bound + rel * (h.abs() + ah + n.abs() * ahn)) / sd + tiny
    R = x.shape[0]
    dw, db = (dy * n).sum(0), dy.sum(0)
    dwb = up * dw.abs() + (R + 8) * E * (dy * n).abs().sum(0) + (dy.abs() * nb).sum(0) + tp
    dbb = up * db.abs() + (R + 8) * E * dy.abs().sum(0) + tp
    got["dx"] = (dx.reshape(*lead, N), dxb.reshape(*lead, N))
    got["dweight"], got["dbias"] = (dw, dwb), (db, dbb)
    return got


def dense_bias(table, q_len, k_len, q_start, max_distance, bidirectional, dy=None):
    u, tiny = U[table.dtype], TINY[table.dtype]
    nb, H = table.shape
    low = -(q_start + q_len)
    known = bucket_tensor(low, k_len - q_start, nb, max_distance, bidirectional)
    i, j = torch.arange(q_len)[:, None], torch.arange(k_len)[None, :]
    at = known[j - (q_start + i) - low].to(table.device)
    out = table.double()[at].permute(2, 0, 1)
    got = {"out": (out, torch.zeros_like(out))}
    if dy is not None:
        d, mag = (torch.zeros(H, nb, dtype=torch.float64, device=table.device) for _ in range(2))
        flat = at.reshape(-1)
        d.index_add_(1, flat, dy.double().reshape(H, -1))
        mag.index_add_(1, flat, dy.double().abs().reshape(H, -1))
        got["dtable"] = (d.t(), (u * d.abs() + q_len * k_len * E * mag).t() + tiny)
    return got


def attention(q, k, v, *, scale=None, causal=False, prefix=None, softcap=0.0, table=None, max_distance=128,
              bidirectional=True, slopes=None, q_docs=None, k_docs=None, k_lens=None, q_start=None, dy=None):
    """{name: (value, bound)}; one batch entry and head at a time."""
    u, tiny = U[q.dtype], TINY[q.dtype]
    B, Tq, H, D = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    dev = q.device

    def new(t):
        return torch.zeros(t.shape, dtype=torch.float64, device=dev)

    out, ob = new(q), new(q)
    lse = torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device=dev)
    lb = torch.zeros_like(lse)
    dq, dqb, dk, dkb, dv, dvb = new(q), new(q), new(k), new(k), new(v), new(v)
    if table is not None:
        nb = table.shape[0]
        dt, dtb = new(table), new(table)
        known = bucket_tensor(-max_distance, max_distance, nb, max_distance, bidirectional).to(dev)
    for b in range(B):
        n = Tk if k_lens is None else max(0, min(Tk, int(k_lens[b])))
        if q_start is None:
            s0 = n - Tq
        else:
            s0 = int(q_start[b]) if isinstance(q_start, torch.Tensor) else int(q_start)
        o = torch.arange(Tk, device=dev)[None, :] - (s0 + torch.arange(Tq, device=dev))[:, None]
        seen = (torch.arange(Tk, device=dev) < n)[None, :].expand(Tq, Tk)
        if causal:
            ok = o <= 0
            if prefix is not None:
                ok = ok | (torch.arange(Tk, device=dev) < int(prefix[b]))[None, :]
            seen = seen & ok
        if q_docs is not None:
            seen = seen & (q_docs[b][:, None] == k_docs[b][None, :]) & (q_docs[b] >= 0)[:, None]
        any_q, any_k = seen.any(1), seen.any(0)
        for h in range(H):
            g = h // (H // Hk)
            # what nothing sees is never used
            K = torch.where(any_k[:, None], k[b, :, g].double(), 0.0)
            V = torch.where(any_k[:, None], v[b, :, g].double(), 0.0)
            Q = torch.where(any_q[:, None], q[b, :, h].double(), 0.0)
            z = scale * (Q @ K.T)
            mag = abs(scale) * (Q.abs() @ K.abs().T)
            slope = torch.ones_like(z)
            if softcap:
                t = torch.tanh(z / softcap)
                slope, z = 1 - t * t, softcap * t
            if table is not None:
                at = known[o.clamp(-max_distance, max_distance) + max_distance]
                z = z + table[:, h].double()[at]
            if slopes is not None:
                z = z - slopes[h].double() * o.abs()
            z = z.masked_fill(~seen, -math.inf)
            L = torch.logsumexp(z, 1)
            p = torch.where(any_q[:, None], torch.exp(z - torch.where(any_q, L, 0.0)[:, None]), 0.0)
            zmag = torch.where(seen, z.abs(), 0.0)
            # a score is off by its product's rounding, and by the rounding of
            # scaled, capped and biased values and of exp's argument
            eps = ((D + 32) * E * torch.where(seen, mag, 0.0).amax(1, keepdim=True)
                   + 32 * E * zmag.amax(1, keepdim=True) + 2.0 ** -20) if Tk else torch.zeros(Tq, 1, device=dev)
            n_sum = (Tk + 16) * E
            up = u if u > E else 0.0  # weights are rounded to the type where products are of that type
            rel = eps + n_sum + up  # of a weight p
            out[b, :, h] = p @ V
            ob[b, :, h] = u * out[b, :, h].abs() + 2 * rel * (p @ V.abs()) + tiny
            lse[b, h] = L
            lb[b, h] = 2 * eps[:, 0] + n_sum + 4 * E * torch.where(any_q, L.abs(), 0.0)
            if dy is None:
                continue
            G = torch.where(any_q[:, None], dy[b, :, h].double(), 0.0)
            dp = G @ V.T
            delta = (G * out[b, :, h]).sum(1, keepdim=True)
            ds = p * (dp - delta)
            # delta from the rounded output; products of dp; the weight itself
            dmag = (G.abs() * (ob[b, :, h] + (D + 4) * E * out[b, :, h].abs())).sum(1, keepdim=True)
            err = p * (2 * rel * (dp.abs() + delta.abs()) + (D + 4) * E * (G.abs() @ V.abs().T) + dmag) + tiny
            dv[b, :, g] += p.T @ G
            many = (Tq * (H // Hk) + 16) * E
            dvb[b, :, g] += (2 * rel * p).T @ G.abs() + many * (p.T @ G.abs())
            if table is not None:
                flat = at.reshape(-1)
                dt[:, h].index_add_(0, flat, ds.reshape(-1))
                dtb[:, h].index_add_(0, flat, (err + (B * Tq * Tk) * E * ds.abs()).reshape(-1))
            # near the cap 1 - tanh^2 loses the error of tanh, 8 e
            dz, dze = ds * slope, err * slope + (8 * E + (eps if softcap else 0.0)) * ds.abs()
            dq[b, :, h] = scale * (dz @ K)
            dqb[b, :, h] = u * dq[b, :, h].abs() + abs(scale) * (dze + (up + n_sum) * dz.abs()) @ K.abs() + tiny
            dk[b, :, g] += scale * (dz.T @ Q)
            dkb[b, :, g] += abs(scale) * ((dze + (up + many) * dz.abs()).T @ Q.abs())
    got = {"out": (out, ob), "lse": (lse, lb)}
    if dy is not None:
        got |= {"dq": (dq, dqb), "dk": (dk, dkb + u * dk.abs() + tiny), "dv": (dv, dvb + u * dv.abs() + tiny)}
        if table is not None:
            ut = U[table.dtype]
            got["dtable"] = (dt, dtb + ut * dt.abs() + TINY[table.dtype])
    return got
