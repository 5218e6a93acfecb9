"""Cases of the frame-encoder operators: layer norm, the learned relative
position bias, and attention over frames whose scores are capped, biased by
distance and masked by recording.

Every case has two forms of the same pass: elementary torch operations in 32
bits, rounded once at the end (`own` False), and the package's own calls
(`own` True). `exact` gives the same outputs from the definitions in 64 bits.

The sizes are those of the mel spectrogram's configurations: 101 frames are one
second at hop 160, 129 the 2 s recordings of the power-of-two configuration,
1292 the 30 s of music, 3001 the 30 s of speech, 360001 an hour of speech.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ITEM = {"f32": 4, "f16": 2, "bf16": 2}


def _norm(name, rows, width, dtype, train):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "train": train}


def _bias(name, heads, q_len, k_len, buckets, max_distance, both_ways, dtype, train):
    return {"name": name, "op": "bias", "heads": heads, "q_len": q_len, "k_len": k_len, "buckets": buckets,
            "max_distance": max_distance, "both_ways": both_ways, "dtype": dtype, "train": train}


def _attention(name, batch, q_len, k_len, heads, kv_heads, dim, dtype, train=False, causal=False, prefix=0, cap=0.0,
               bias="none", buckets=32, max_distance=128, docs=0, ragged=False):
    return {"name": name, "op": "attention", "batch": batch, "q_len": q_len, "k_len": k_len, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "train": train, "causal": causal, "prefix": prefix,
            "cap": cap, "bias": bias, "buckets": buckets, "max_distance": max_distance, "docs": docs,
            "ragged": ragged}


def listed():
    return [
        # the norm before a block, one second of speech arriving live: latency
        _norm("norm-second", 101, 512, "bf16", False),
        # frames normalised over their 80 mel bins, 64 recordings of 129 frames, trained
        _norm("norm-mels", 64 * 129, 80, "f32", True),
        # a block's norm in training on 64 music recordings of 1292 frames
        _norm("norm-music", 64 * 1292, 1024, "bf16", True),
        # the dense bias of one second of frames, for a caller's own scores: latency
        _bias("bias-second", 8, 101, 101, 32, 128, True, "f32", False),
        # the dense bias of 30 s of speech and its gradient, 320 buckets up to 800 frames
        _bias("bias-speech", 16, 3001, 3001, 320, 800, True, "bf16", True),
        # one new frame against the second before it: latency
        _attention("step-second", 1, 1, 101, 8, 8, 64, "f16", bias="buckets"),
        # one new token for each of 64 streams, caches of up to 30 s filled unevenly, heads that share keys
        _attention("step-streams", 64, 1, 3001, 16, 4, 128, "bf16", bias="slopes", ragged=True),
        # four new tokens against an hour of frames, capped scores
        _attention("step-hour", 1, 4, 360001, 8, 2, 64, "f16", cap=30.0, causal=True),
        # a training step on a few short recordings in 32 bits, head size 40
        _attention("train-short", 2, 129, 129, 4, 4, 40, "f32", train=True, bias="buckets", docs=2),
        # encoding 8 recordings of 30 s, no gradient
        _attention("encode-speech", 8, 3001, 3001, 16, 16, 128, "bf16", ragged=True),
        # training an encoder: rows of 30 s, each packed with three recordings, learned bias by distance
        _attention("train-packed", 8, 3001, 3001, 8, 8, 64, "bf16", train=True, bias="buckets", buckets=320,
                   max_distance=800, docs=3),
        # training a frame predictor: causal after a prefix, capped scores, linear bias, heads that share keys
        _attention("train-causal", 8, 1292, 1292, 16, 4, 128, "f16", train=True, causal=True, prefix=129, cap=30.0,
                   bias="slopes"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "bias", "step", "encode", "train", "train"])
    if kind == "norm":
        rows, width = _log(rng, 1, 64 * 1292), _log(rng, 8, 4096)
        rows = max(1, min(rows, 64 * 1292 * 1024 // width))
        c = _norm("", rows, width, rng.choice(["f32", "f16", "bf16"]), rng.random() < 0.6)
        if c["dtype"] == "f32":
            c["rows"] = max(1, rows // 2)
    elif kind == "bias":
        heads, t = rng.choice([1, 4, 8, 12, 16]), _log(rng, 1, 3001)
        far = rng.choice([32, 128, 800])
        c = _bias("", heads, max(1, t - rng.choice([0, 0, 1, 37])), t, rng.choice([32, 64, 320] if far == 800 else [16, 32]),
                  far, rng.random() < 0.6, rng.choice(["f32", "f16", "bf16"]), rng.random() < 0.6)
        if c["dtype"] == "f32":
            c["heads"] = max(1, heads // 2)
    elif kind == "step":
        batch, k_len = _log(rng, 1, 64), _log(rng, 1, 360001)
        kv = rng.choice([1, 2, 4, 8])
        heads, dim = kv * rng.choice([1, 2, 4]), rng.choice([64, 64, 128, 80])
        k_len = max(1, min(k_len, 64 * 3001 * 4 * 128 // (batch * kv * dim)))
        bias = rng.choice(["none", "buckets", "slopes"])
        c = _attention("", batch, rng.choice([1, 1, 1, 2, 4]), k_len, heads, kv, dim, rng.choice(["f16", "bf16"]),
                       causal=rng.random() < 0.5, cap=rng.choice([0.0, 0.0, 30.0]), bias=bias,
                       ragged=rng.random() < 0.5)
        c["q_len"] = min(c["q_len"], k_len)
    else:
        train = kind == "train"
        dtype = rng.choice(["f32", "f16", "bf16", "bf16", "f16"])
        kv = rng.choice([1, 2, 4, 8])
        heads, dim = kv * rng.choice([1, 1, 2, 4]), rng.choice([40, 80, 64] if dtype == "f32" else [64, 128, 64, 128, 80])
        t = _log(rng, 5, 320 if dtype == "f32" else 3001)
        batch = _log(rng, 1, 8)
        most = 1.3e10 if train else 3e10  # pairs times head size, as many as the largest listed cases have
        t = min(t, int(math.sqrt(most / (heads * dim))))
        batch = max(1, min(batch, int(most / (heads * t * t * dim))))
        far = rng.choice([128, 800])
        c = _attention("", batch, t, t, heads, kv, dim, dtype, train=train, causal=rng.random() < 0.4,
                       cap=rng.choice([0.0, 0.0, 30.0]), bias=rng.choice(["none", "buckets", "slopes"]),
                       buckets=320 if far == 800 else 32, max_distance=far,
                       docs=rng.choice([0, 0, 2, 3, 5]) if t > 20 else 0)
        if c["causal"] and rng.random() < 0.5:
            c["prefix"] = rng.randint(1, t)
        if not c["docs"]:
            c["ragged"] = rng.random() < 0.5
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# what belongs to a case whatever the seed: how long its recordings are

def _lengths(case):
    """Frames in use in each row of the batch, [B]."""
    if not case["ragged"]:
        return np.full(case["batch"], case["k_len"], np.int64)
    r = np.random.default_rng([case["batch"], case["k_len"], 5])
    return r.integers((case["k_len"] + 1) // 2, case["k_len"] + 1, case["batch"])


def _starts(case):
    """The key place of each row's first query, [B]: whole rows attend to
    themselves, shorter ones are the newest frames of the row."""
    return _lengths(case) - case["q_len"] if case["q_len"] < case["k_len"] else np.zeros(case["batch"], np.int64)


def _documents(case):
    """Which recording each frame belongs to, [B, T]; -1 is padding."""
    r = np.random.default_rng([case["batch"], case["k_len"], case["docs"]])
    ids = np.full((case["batch"], case["k_len"]), -1, np.int32)
    for row in ids:
        cuts = np.sort(r.integers(1, case["k_len"], case["docs"]))
        for n, (a, b) in enumerate(zip([0, *cuts[:-1]], cuts)):
            row[a:b] = n
    return ids


def _pairs(case):
    """Pairs of a query and a key that it may see, over the batch."""
    i = np.arange(case["q_len"], dtype=np.int64)
    total = 0
    lens, starts = _lengths(case), _starts(case)
    docs = _documents(case) if case["docs"] else None
    for b in range(case["batch"]):
        if docs is not None:
            ids = docs[b]
            first = np.searchsorted(np.where(ids < 0, 1 << 30, ids), ids, "left")
            last = np.searchsorted(np.where(ids < 0, 1 << 30, ids), ids, "right")
            last = np.where(ids < 0, first, last)
        else:
            first, last = np.zeros_like(i), np.full_like(i, lens[b])
        if case["causal"]:
            place = i + starts[b]
            last = np.minimum(last, np.maximum(place + 1, case["prefix"]))
        total += int(np.maximum(last - first, 0).sum())
    return total


def work(case):
    item = _ITEM[case["dtype"]]
    if case["op"] == "norm":
        n, w = case["rows"] * case["width"], case["width"]
        if case["train"]:  # in: x, dy, weight, bias; out: y, dx, dweight, dbias
            return {"bytes": item * (4 * n + 4 * w), "flops": 18 * n}
        return {"bytes": item * (2 * n + 2 * w), "flops": 8 * n}
    if case["op"] == "bias":
        n, t = case["heads"] * case["q_len"] * case["k_len"], case["buckets"] * case["heads"]
        return {"bytes": item * ((2 * n + 2 * t) if case["train"] else (n + t)), "flops": n if case["train"] else 0}
    q = case["batch"] * case["q_len"] * case["heads"] * case["dim"]
    kv = 2 * int(_lengths(case).sum()) * case["kv_heads"] * case["dim"]
    table = case["buckets"] * case["heads"] if case["bias"] == "buckets" else 0
    product = 2 * _pairs(case) * case["heads"] * case["dim"]
    if case["train"]:  # in: q, k, v, dout, table; out: out, dq, dk, dv, dtable
        return {"bytes": item * (4 * q + 2 * kv + 2 * table), "flops": 7 * product}
    return {"bytes": item * (2 * q + kv + table), "flops": 2 * product}


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale + shift).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        # activations have a mean of their own in each frame; weights stay near one
        x = torch.randn(case["rows"], case["width"], device="cuda", generator=g) * 1.5
        x += torch.randn(case["rows"], 1, device="cuda", generator=g)
        s["x"] = x.to(dtype)
        s["weight"] = normal(case["width"], scale=0.2, shift=1.0)
        s["bias"] = normal(case["width"], scale=0.2)
        if case["train"]:
            s["dy"] = normal(case["rows"], case["width"])
            for n in ("x", "weight", "bias"):
                s[n].requires_grad_()
        return s
    if case["op"] == "bias":
        s["table"] = normal(case["buckets"], case["heads"])
        if case["train"]:
            s["dy"] = normal(case["heads"], case["q_len"], case["k_len"])
            s["table"].requires_grad_()
        return s
    B, Tq, Tk, H, Hk, D = (case[n] for n in ("batch", "q_len", "k_len", "heads", "kv_heads", "dim"))
    if Tq == Tk:
        # one projection gives all three: views of one buffer
        qkv = normal(B, Tq, H + 2 * Hk, D)
        s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:]
    else:
        s["q"] = normal(B, Tq, H, D)
        s["k"], s["v"] = normal(B, Tk, Hk, D), normal(B, Tk, Hk, D)
    if case["docs"]:
        s["documents"] = torch.from_numpy(_documents(case)).cuda()
    if case["ragged"]:
        s["lengths"] = torch.from_numpy(_lengths(case).astype(np.int32)).cuda()
    if case["prefix"]:
        s["prefix"] = torch.full((B,), case["prefix"], dtype=torch.int32, device="cuda")
    if case["bias"] == "buckets":
        s["table"] = normal(case["buckets"], H)
    if case["bias"] == "slopes":
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)
    if case["train"]:
        s["dy"] = normal(B, Tq, H, D)
        for n in ("q", "k", "v", "table"):
            if n in s:
                s[n] = s[n].detach().requires_grad_()
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    with torch.no_grad():
        if case["op"] == "norm":
            return _plain_norm(s, case)
        if case["op"] == "bias":
            return _plain_bias(s, case)
        return _plain_attention(s, case)


def _run_own(s, case):
    from mel_spectrogram_gb300 import attention, layer_norm, relative_bias

    if case["op"] == "norm":
        out = layer_norm(s["x"], s["weight"], s["bias"], eps=1e-5)
        names = ("x", "weight", "bias")
    elif case["op"] == "bias":
        out = relative_bias(s["table"], case["q_len"], case["k_len"], max_distance=case["max_distance"],
                            bidirectional=case["both_ways"])
        names = ("table",)
    else:
        out = attention(s["q"], s["k"], s["v"], causal=case["causal"], prefix=s.get("prefix"), softcap=case["cap"],
                        table=s.get("table"), max_distance=case["max_distance"], slopes=s.get("slopes"),
                        q_docs=s.get("documents"), k_docs=s.get("documents"), k_lens=s.get("lengths"),
                        q_start=0 if case["q_len"] == case["k_len"] else None)
        names = ("q", "k", "v", "table") if "table" in s else ("q", "k", "v")
    if not case["train"]:
        return {"out": out}
    grads = torch.autograd.grad(out, [s[n] for n in names], s["dy"])
    return {"out": out.detach(), **{"d" + n: x for n, x in zip(names, grads)}}


def _plain_norm(s, case):
    dtype = _DTYPES[case["dtype"]]
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    n = c * rstd
    out = {"out": (n * w + b).to(dtype)}
    if case["train"]:
        dy = s["dy"].float()
        h = dy * w
        dx = rstd * (h - h.mean(-1, keepdim=True) - n * (h * n).mean(-1, keepdim=True))
        out["dx"] = dx.to(dtype)
        out["dweight"] = (dy * n).sum(0).to(dtype)
        out["dbias"] = dy.sum(0).to(dtype)
    return out


def _buckets(offset, buckets, max_distance, both_ways):
    """The bucket of key place minus query place."""
    side = buckets // 2 if both_ways else buckets
    n = offset.abs() if both_ways else (-offset).clamp(min=0)
    exact = side // 2
    # the nudge keeps the powers that land on a whole number from rounding below it
    far = torch.log(n.clamp(min=1).double() / exact) / math.log(max_distance / exact) * (side - exact) + 1e-9
    n = torch.where(n < exact, n, (exact + far.floor().long()).clamp(max=side - 1))
    return n + side * (offset > 0) if both_ways else n


def _diagonals(z):
    """Sums of [..., Tq, Tk] over equal j - i, from 1 - Tq to Tk - 1."""
    Tq, Tk = z.shape[-2:]
    z = torch.nn.functional.pad(z.flip(-2), (0, Tq)).flatten(-2)[..., :Tq * (Tk + Tq - 1)]
    return z.unflatten(-1, (Tq, Tk + Tq - 1)).sum(-2)


def _plain_bias(s, case):
    dtype = _DTYPES[case["dtype"]]
    i = torch.arange(case["q_len"], device="cuda")[:, None] + (case["k_len"] - case["q_len"])
    j = torch.arange(case["k_len"], device="cuda")[None, :]
    at = _buckets(j - i, case["buckets"], case["max_distance"], case["both_ways"])
    out = {"out": s["table"].t()[:, at].contiguous()}
    if case["train"]:
        offset = torch.arange(1 - case["q_len"], case["k_len"], device="cuda") - (case["k_len"] - case["q_len"])
        at = _buckets(offset, case["buckets"], case["max_distance"], case["both_ways"])
        d = torch.zeros(case["heads"], case["buckets"], device="cuda")
        d.index_add_(1, at, _diagonals(s["dy"].float()))
        out["dtable"] = d.t().to(dtype)
    return out


def _plain_attention(s, case):
    dtype = _DTYPES[case["dtype"]]
    B, Tq, Tk, H, Hk, D = (case[n] for n in ("batch", "q_len", "k_len", "heads", "kv_heads", "dim"))
    G, scale = H // Hk, 1.0 / math.sqrt(D)
    q = s["q"].float().transpose(1, 2).reshape(B, Hk, G, Tq, D)
    k = s["k"].float().transpose(1, 2).reshape(B, Hk, 1, Tk, D)
    v = s["v"].float().transpose(1, 2).reshape(B, Hk, 1, Tk, D)
    z = q @ k.transpose(-1, -2) * scale
    cap = case["cap"]
    if cap:
        t = torch.tanh(z / cap)
        z = cap * t
    lens = s["lengths"] if "lengths" in s else torch.full((B,), Tk, device="cuda")
    start = lens - Tq if Tq < Tk else torch.zeros_like(lens)
    place = torch.arange(Tq, device="cuda")[None, :] + start[:, None]  # [B, Tq]
    j = torch.arange(Tk, device="cuda")
    offset = j - place[:, :, None]  # [B, Tq, Tk]
    if case["bias"] == "buckets":
        at = _buckets(offset, case["buckets"], case["max_distance"], True)
        z = z + s["table"].float()[at].permute(0, 3, 1, 2).reshape(B, Hk, G, Tq, Tk)
    if case["bias"] == "slopes":
        z = z - s["slopes"].reshape(1, Hk, G, 1, 1) * offset.abs().float()[:, None, None]
    seen = (j < lens[:, None])[:, None, :].expand(B, Tq, Tk)
    if case["causal"]:
        near = offset <= 0
        if case["prefix"]:
            near = near | (j < s["prefix"][:, None])[:, None, :]
        seen = seen & near
    if case["docs"]:
        ids = s["documents"]
        seen = seen & (ids[:, :, None] == ids[:, None, :]) & (ids >= 0)[:, :, None]
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = p @ v
    out = {"out": o.reshape(B, H, Tq, D).transpose(1, 2).to(dtype)}
    if case["train"]:
        do = s["dy"].float().transpose(1, 2).reshape(B, Hk, G, Tq, D)
        dv = (p.transpose(-1, -2) @ do).sum(2)
        dz = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        if case["bias"] == "buckets":
            at = _buckets(torch.arange(1 - Tq, Tk, device="cuda") - start[:, None], case["buckets"],
                          case["max_distance"], True)
            sums = _diagonals(dz.reshape(B, H, Tq, Tk)).transpose(0, 1).reshape(H, -1)
            d = torch.zeros(H, case["buckets"], device="cuda")
            d.index_add_(1, at.reshape(-1), sums)
        if cap:
            dz = dz * (1 - t * t)
        dq = (dz @ k) * scale
        dk = (dz.transpose(-1, -2) @ q).sum(2) * scale
        out["dq"] = dq.reshape(B, H, Tq, D).transpose(1, 2).to(dtype)
        out["dk"] = dk.transpose(1, 2).to(dtype)
        out["dv"] = dv.transpose(1, 2).to(dtype)
        if case["bias"] == "buckets":
            out["dtable"] = d.t().to(dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _bucket_map(low, high, buckets, max_distance, both_ways):
    """Buckets of the offsets low..high in whole numbers: beyond the exact half
    of a side, n's bucket is the last m with n^L >= e^(L-m) * M^m."""
    side = buckets // 2 if both_ways else buckets
    e, L = side // 2, side - side // 2

    def of(n):
        if n < e:
            return n
        m = 0
        while m < L - 1 and n ** L >= e ** (L - m - 1) * max_distance ** (m + 1):
            m += 1
        return e + m

    known = [of(n) for n in range(max_distance + 1)]

    def bucket(d):
        if both_ways:
            return known[min(abs(d), max_distance)] + (side if d > 0 else 0)
        return known[min(max(-d, 0), max_distance)]

    return np.array([bucket(d) for d in range(low, high + 1)], np.int64)


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "norm":
            x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
            var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
            sd = (var + 1e-5).sqrt()
            n = (x - mean) / sd
            out = {"out": torch.addcmul(b, n, w)}
            if case["train"]:
                dy, N = s["dy"].double(), case["width"]
                h = dy * w
                out["dx"] = (N * h - h.sum(-1, keepdim=True) - n * (h * n).sum(-1, keepdim=True)) / (N * sd)
                out["dweight"] = torch.einsum("rw,rw->w", dy, n)
                out["dbias"] = torch.einsum("rw->w", dy)
            return out
        if case["op"] == "bias":
            Tq, Tk = case["q_len"], case["k_len"]
            known = torch.from_numpy(_bucket_map(-(Tk - 1), Tq + Tk, case["buckets"], case["max_distance"],
                                                 case["both_ways"])).cuda()
            out = torch.empty(case["heads"], Tq, Tk, device="cuda", dtype=torch.float64)
            table = s["table"].double()
            d = torch.zeros_like(table)
            for i in range(Tq):
                at = known[Tq - 1 - i:Tq - 1 - i + Tk]
                out[:, i] = table[at].t()
                if case["train"]:
                    d.index_add_(0, at, s["dy"][:, i].double().t())
            return {"out": out, "dtable": d} if case["train"] else {"out": out}
        return _exact_attention(s, case)


def _exact_attention(s, case):
    B, Tq, Tk, H, Hk, D = (case[n] for n in ("batch", "q_len", "k_len", "heads", "kv_heads", "dim"))
    if B * H * Tq * Tk * D * (5 if case["train"] else 2) > 6e12:
        return None
    lens, starts = _lengths(case), _starts(case)
    docs = _documents(case) if case["docs"] else None
    scale, cap = D ** -0.5, case["cap"]
    new = lambda like: torch.zeros(like.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out, dq, dk, dv = new(s["q"]), new(s["q"]), new(s["k"]), new(s["v"])
    if case["bias"] == "buckets":
        known = torch.from_numpy(_bucket_map(-(Tk + Tq), Tk + Tq, case["buckets"], case["max_distance"], True)).cuda()
        dtable = new(s["table"])
    for b in range(B):
        n = int(lens[b])
        place = torch.arange(Tq, device="cuda") + int(starts[b])
        delta = torch.arange(n, device="cuda")[None, :] - place[:, None]
        blind = torch.zeros(Tq, n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            blind |= delta > 0
            blind[:, :case["prefix"]] = False
        if docs is not None:
            ids = torch.from_numpy(docs[b]).cuda()
            blind |= ids[:, None] != ids[None, :n]
            blind[ids < 0] = True
        for h in range(H):
            g = h // (H // Hk)
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :n, g].double(), s["v"][b, :n, g].double()
            z = scale * (q @ k.T)
            slope = 1.0
            if cap:
                t = torch.tanh(z / cap)
                z, slope = cap * t, 1 - t ** 2
            if case["bias"] == "buckets":
                at = known[delta + (Tk + Tq)]
                z = z + s["table"][:, h].double()[at]
            elif case["bias"] == "slopes":
                z = z - s["slopes"][h].double() * delta.abs()
            z[blind] = -math.inf
            p = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
            out[b, :, h] = p @ v
            if case["train"]:
                do = s["dy"][b, :, h].double()
                dv[b, :n, g] += p.T @ do
                dp = do @ v.T
                dz = p * (dp - (p * dp).sum(-1, keepdim=True))
                if case["bias"] == "buckets":
                    dtable[:, h].index_add_(0, at.reshape(-1), dz.reshape(-1))
                dz = dz * slope * scale
                dq[b, :, h] = dz @ k
                dk[b, :n, g] += dz.T @ q
    if not case["train"]:
        return {"out": out}
    got = {"out": out, "dq": dq, "dk": dk, "dv": dv}
    if case["bias"] == "buckets":
        got["dtable"] = dtable
    return got
