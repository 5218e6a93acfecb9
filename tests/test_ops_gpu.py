"""Layer norm, the position bias and attention against their definitions in 64
bits (ops_reference), element by element within derived bounds."""
from __future__ import annotations

import math

import pytest
import torch

from tests import ops_reference as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300 import ops

    return ops


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale + shift).to(dtype)


# ---------------------------------------------------------------------------
# layer norm

NORM_SHAPES = [(1, 1), (1, 2), (3, 5), (101, 80), (7, 128), (129, 512), (33, 1000), (5, 1111), (2, 2048), (3, 2049),
               (4, 4096), (2, 8192), (2, 12000), (700, 256), (3, 20001)]


def run_norm(ops, x, w, b, eps, dy, affine=True):
    x = x.detach().requires_grad_()
    leaves = [x]
    if w is not None:
        w = w.detach().requires_grad_()
        leaves.append(w)
    if b is not None:
        b = b.detach().requires_grad_()
        leaves.append(b)
    y = ops.layer_norm(x, w, b, eps=eps)
    grads = torch.autograd.grad(y, leaves, dy)
    return y, grads


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", NORM_SHAPES)
def test_norm(ops, rows, width, dtype):
    g = gen(rows * 31 + width)
    x = randn(g, rows, width, dtype=dtype, scale=1.5, shift=0.7)
    w, b = randn(g, width, dtype=dtype, scale=0.2, shift=1.0), randn(g, width, dtype=dtype)
    dy = randn(g, rows, width, dtype=dtype)
    want = ref.norm(x, w, b, 1e-5, dy)
    y, (dx, dw, db) = run_norm(ops, x, w, b, 1e-5, dy)
    for name, got in (("out", y), ("dx", dx), ("dweight", dw), ("dbias", db)):
        assert got.dtype == dtype
        ref.close(got, *want[name], f"{name} {rows}x{width} {dtype}")
    plain = ops.layer_norm(x, w, b, eps=1e-5)  # no graph: the same bits
    assert torch.equal(plain, y)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_norm_wide_parameters_and_none(ops, dtype):
    g = gen(3)
    x, dy = randn(g, 37, 384, dtype=dtype), randn(g, 37, 384, dtype=dtype)
    w, b = randn(g, 384, shift=1.0), randn(g, 384)
    want = ref.norm(x, w, b, 1e-3, dy)
    y, (dx, dw, db) = run_norm(ops, x, w, b, 1e-3, dy)
    assert dw.dtype == F32 and db.dtype == F32
    for name, got in (("out", y), ("dx", dx), ("dweight", dw), ("dbias", db)):
        ref.close(got, *want[name], name)
    want = ref.norm(x, None, None, 1e-3, dy)
    y, (dx,) = run_norm(ops, x, None, None, 1e-3, dy)
    ref.close(y, *want["out"], "out")
    ref.close(dx, *want["dx"], "dx")


def test_norm_layouts(ops):
    g = gen(4)
    base = randn(g, 6, 9, 200, dtype=BF16)
    w, b = randn(g, 200, dtype=BF16), randn(g, 200, dtype=BF16)
    views = [base[:, 1:5], base[:, :, 3:131], base.transpose(0, 1), base.transpose(1, 2), base[::2, ::3],
             base[:1].expand(5, 9, 200), base[0, 0], base[0, :1]]
    for x in views:
        n = x.shape[-1]
        ww, bb = (w[:n], b[:n]) if n <= 200 else (w, b)
        dy = torch.randn(x.shape, device="cuda", generator=g).to(BF16)
        for d in (dy, dy.expand(x.shape), dy.transpose(0, -1).contiguous().transpose(0, -1) if dy.dim() > 1 else dy):
            want = ref.norm(x, ww, bb, 1e-5, d)
            y, (dx, dw, db) = run_norm(ops, x, ww, bb, 1e-5, d)
            for name, got in (("out", y), ("dx", dx), ("dweight", dw), ("dbias", db)):
                ref.close(got, *want[name], f"{name} {tuple(x.shape)} {x.stride()}")


def test_norm_constant_and_large_rows(ops):
    # a constant row has variance 0; a large mean must not eat the variance
    x = torch.full((2, 96), 3.0, device="cuda")
    y = ops.layer_norm(x)
    assert torch.equal(y, torch.zeros_like(y))
    g = gen(5)
    x = randn(g, 8, 640, scale=1.0, shift=1000.0)
    ref.close(ops.layer_norm(x), *ref.norm(x, None, None, 1e-5)["out"], "large mean")


def test_norm_empty_and_nonfinite(ops):
    x = torch.empty(0, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    y = ops.layer_norm(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), torch.empty_like(y))
    assert y.shape == (0, 64) and dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w))
    x = torch.randn(3, 64, device="cuda")
    x[1, 5] = math.nan
    y = ops.layer_norm(x)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()


def test_norm_differences(ops):
    # directional differences of the 64-bit definition against the kernel's gradient
    g = gen(6)
    x, dy = randn(g, 20, 100), randn(g, 20, 100)
    w, b = randn(g, 100, shift=1.0), randn(g, 100)
    _, grads = run_norm(ops, x, w, b, 1e-5, dy)
    for n, t in enumerate((x, w, b)):
        step = randn(g, *t.shape)

        def loss(s):
            args = [a.double() for a in (x, w, b)]
            args[n] = args[n] + s * step.double()
            c = args[0] - args[0].mean(-1, keepdim=True)
            y = c / ((c * c).mean(-1, keepdim=True) + 1e-5).sqrt() * args[1] + args[2]
            return float((y * dy.double()).sum())

        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = float((grads[n].double() * step.double()).sum())
        scale = float((grads[n].double().abs() * step.double().abs()).sum())
        # central differences of step 1e-5 err by its square; the gradients by about 200 roundings
        assert abs(got - slope) <= scale * (200 * ref.E + 1e-7)


def test_norm_same_bits_and_streams(ops):
    g = gen(7)
    x, dy = randn(g, 3000, 512, dtype=BF16), randn(g, 3000, 512, dtype=BF16)
    w, b = randn(g, 512, dtype=BF16), randn(g, 512, dtype=BF16)
    first = run_norm(ops, x, w, b, 1e-5, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run_norm(ops, x, w, b, 1e-5, dy)
    side.synchronize()
    assert torch.equal(first[0], again[0])
    for a, c in zip(first[1], again[1]):
        assert torch.equal(a, c)


# ---------------------------------------------------------------------------
# buckets and the dense bias

@pytest.mark.parametrize("config", [(32, 128, True), (32, 128, False), (320, 800, True), (4, 2, True), (2, 2, False),
                                    (16, 128, True), (64, 2048, True), (7, 100, False), (4096, 2048, True)])
def test_bucket_map(ops, config):
    nb, far, both = config
    got = ops.bucket_map(nb, far, both)
    want = ref.bucket_tensor(-far, far, nb, far, both)
    assert torch.equal(got.long(), want)


BIAS = [
    (8, 101, 101, None, 32, 128, True), (1, 1, 1, None, 32, 128, True), (3, 1, 257, None, 32, 128, True),
    (2, 5, 3, None, 16, 100, False), (4, 300, 517, None, 320, 800, True), (5, 517, 300, 0, 32, 40, True),
    (2, 33, 64, -1000, 32, 128, True), (2, 33, 64, 10 ** 12, 32, 128, False), (1, 2100, 70, 3, 64, 900, True),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", BIAS)
def test_relative_bias(ops, case, dtype):
    H, Tq, Tk, q_start, nb, far, both = case
    g = gen(Tq + Tk)
    table = randn(g, nb, H, dtype=dtype).requires_grad_()
    dy = randn(g, H, Tq, Tk, dtype=dtype)
    start = Tk - Tq if q_start is None else max(-10 ** 6, min(10 ** 6, q_start))
    want = ref.dense_bias(table.detach(), Tq, Tk, start, far, both, dy)
    out = ops.relative_bias(table, Tq, Tk, q_start, max_distance=far, bidirectional=both)
    (d,) = torch.autograd.grad(out, table, dy)
    ref.close(out, *want["out"], f"out {case}")
    ref.close(d, *want["dtable"], f"dtable {case}")


def test_relative_bias_broadcast_gradient(ops):
    # added to a batch of scores: the gradient arrives summed, or expanded from one value
    g = gen(9)
    table = randn(g, 32, 4).requires_grad_()
    scores = randn(g, 3, 4, 50, 70)
    dy = randn(g, 3, 4, 50, 70)
    out = scores + ops.relative_bias(table, 50, 70)
    (d,) = torch.autograd.grad(out, table, dy)
    ref.close(d, *ref.dense_bias(table.detach(), 50, 70, 20, 128, True, dy.sum(0))["dtable"], "summed")
    out = ops.relative_bias(table, 50, 70)
    (d,) = torch.autograd.grad(out.sum(), table)
    ones = torch.ones(4, 50, 70, device="cuda")
    ref.close(d, *ref.dense_bias(table.detach(), 50, 70, 20, 128, True, ones)["dtable"], "expanded")


def test_relative_bias_empty(ops):
    table = torch.randn(32, 4, device="cuda", requires_grad=True)
    for shape in ((0, 5), (5, 0), (0, 0)):
        out = ops.relative_bias(table, *shape)
        assert out.shape == (4, *shape)
        (d,) = torch.autograd.grad(out.sum(), table)
        assert torch.equal(d, torch.zeros_like(d))


# ---------------------------------------------------------------------------
# attention

def lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def docs_of(T, *rows):
    """One row of ids per list of (id, count) runs; the rest is padding."""
    ids = torch.full((len(rows), T), -1, dtype=torch.int32, device="cuda")
    for r, runs in enumerate(rows):
        at = 0
        for n, count in runs:
            ids[r, at:at + count] = n
            at += count
    return ids


def check_attention(ops, q, k, v, what, dy=None, **kw):
    want = ref.attention(q, k, v, dy=dy, **kw)
    if dy is None:
        out, lse = ops.attention(q, k, v, return_lse=True, **kw)
        ref.close(out, *want["out"], f"out {what}")
        ref.close(lse, *want["lse"], f"lse {what}")
        return out
    names = ["q", "k", "v"]
    leaves = [t.detach().requires_grad_() for t in (q, k, v)]
    if kw.get("table") is not None:
        kw = dict(kw, table=kw["table"].detach().requires_grad_())
        leaves.append(kw["table"])
        names.append("table")
    out, lse = ops.attention(*leaves[:3], return_lse=True, **kw)
    grads = torch.autograd.grad(out, leaves, dy)
    ref.close(out, *want["out"], f"out {what}")
    ref.close(lse, *want["lse"], f"lse {what}")
    for n, d in zip(names, grads):
        ref.close(d, *want["d" + n], f"d{n} {what}")
    return out, grads


# batch, q_len, k_len, heads, kv_heads, dim
SHAPES = [(1, 1, 1, 1, 1, 64), (2, 129, 129, 2, 2, 64), (1, 127, 300, 4, 2, 128), (2, 65, 257, 2, 1, 80),
          (1, 300, 129, 3, 3, 40), (1, 70, 70, 2, 1, 1), (1, 50, 90, 2, 2, 3), (1, 40, 130, 2, 1, 256),
          (3, 1, 517, 8, 2, 64), (2, 4, 1000, 8, 1, 128), (1, 513, 513, 1, 1, 96), (1, 16, 16, 2, 2, 200)]


def make(shape, dtype, seed=0):
    B, Tq, Tk, H, Hk, D = shape
    g = gen(seed + 7 * Tq + Tk + D)
    return (randn(g, B, Tq, H, D, dtype=dtype), randn(g, B, Tk, Hk, D, dtype=dtype),
            randn(g, B, Tk, Hk, D, dtype=dtype), randn(g, B, Tq, H, D, dtype=dtype), g)


OPTIONS = {
    "plain": lambda s, t, g: {},
    "causal": lambda s, t, g: {"causal": True},
    "cap": lambda s, t, g: {"softcap": 5.0, "scale": 0.5},
    "buckets": lambda s, t, g: {"table": randn(g, 32, s[3], dtype=t), "max_distance": 50},
    "slopes": lambda s, t, g: {"slopes": torch.rand(s[3], device="cuda", generator=g), "q_start": 3},
    "all": lambda s, t, g: {"causal": True, "prefix": torch.full((s[0],), 20, dtype=torch.int32, device="cuda"),
                            "softcap": 10.0, "table": randn(g, 320, s[3]), "max_distance": 800,
                            "k_lens": torch.full((s[0],), max(1, s[2] - 3), dtype=torch.int32, device="cuda")},
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_attention(ops, shape, option, dtype):
    q, k, v, dy, g = make(shape, dtype)
    kw = OPTIONS[option](shape, dtype, g)
    check_attention(ops, q, k, v, f"{shape} {option} {dtype}", **kw)
    check_attention(ops, q, k, v, f"{shape} {option} {dtype}", dy=dy, **kw)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("option", ["plain", "causal", "all"])
@pytest.mark.parametrize("Tq", [15, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (3, 3)])
def test_attention_few_queries(ops, heads, kv_heads, Tq, option, dtype):
    # both sides of the limits of the kernel for few queries
    shape = (2, Tq, 700, heads, kv_heads, 64)
    q, k, v, _, g = make(shape, dtype, seed=Tq)
    kw = dict(OPTIONS[option](shape, dtype, g), q_start=lengths(700 - Tq, 40))
    check_attention(ops, q, k, v, f"{shape} {option} {dtype}", **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [40, 64, 128])
def test_attention_documents(ops, dtype, dim):
    T = 400
    q, k, v, dy, g = make((3, T, T, 2, 1, dim), dtype)
    ids = docs_of(T, [(0, 100), (1, 1), (2, 250)], [(5, 128), (5, 128), (7, 144)], [(-1, 30), (3, 64), (2, 65), (3, 20)])
    table = randn(g, 32, 2, dtype=dtype)
    for causal in (False, True):
        check_attention(ops, q, k, v, f"docs causal={causal}", dy=dy, q_docs=ids, k_docs=ids, table=table,
                        causal=causal)
    # ids of the queries and the keys that never meet, in one row
    other = ids.clone()
    other[1] = 9
    out = check_attention(ops, q, k, v, "docs apart", q_docs=ids, k_docs=other)
    assert torch.equal(out[1], torch.zeros_like(out[1]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Tq,Tk", [(130, 130), (1, 300), (5, 300)])
def test_attention_unused_memory(ops, dtype, Tq, Tk):
    # infinities and NaN past the lengths and in padding frames change nothing
    q, k, v, dy, g = make((2, Tq, Tk, 2, 2, 64), dtype)
    lens = lengths(Tk - 70, 0)
    for t in (k, v):
        t[0, Tk - 70:] = math.nan
        t[1] = math.inf
    out, grads = check_attention(ops, q, k, v, "lens", dy=dy, k_lens=lens, q_start=0)
    assert torch.equal(out[1], torch.zeros_like(out[1]))
    for d in grads[1:]:
        assert torch.equal(d[0, Tk - 70:], torch.zeros_like(d[0, Tk - 70:]))
    if Tq == Tk:
        q, k, v, dy, g = make((2, Tq, Tk, 2, 2, 64), dtype)
        ids = docs_of(Tk, [(0, 50), (-1, 20), (1, 30)], [(1, 129)])
        pad = ids < 0
        for t, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (dy, -math.inf)):
            t[pad] = bad
        out, grads = check_attention(ops, q, k, v, "docs", dy=dy, q_docs=ids, k_docs=ids)
        for t in (out, *grads):
            assert torch.equal(t[pad], torch.zeros_like(t[pad]))


def test_attention_masked_scores(ops):
    # a masked key's score may be anything: NaN in k reaches only the rows that see it
    q, k, v, dy, g = make((1, 200, 200, 1, 1, 64), BF16)
    k[0, 150] = math.nan
    out = ops.attention(q, k, v, causal=True)
    assert torch.isfinite(out[0, :150]).all() and torch.isnan(out[0, 150:]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dim", [64, 128, 40])
def test_attention_hidden_values(ops, dtype, bad, dim):
    # recordings side by side, one of them broken: the other's results and
    # gradients are those of the whole batch without the broken one's values
    T = 200
    ids = docs_of(T, [(0, 90), (1, 70), (2, 40)])
    q, k, v, dy, g = make((1, T, T, 2, 1, dim), dtype)
    for causal in (False, True):
        clean = check_attention(ops, q, k, v, "clean", dy=dy, q_docs=ids, k_docs=ids, causal=causal)
        broken = [t.clone() for t in (q, k, v, dy)]
        for t in broken:
            t[:, 90:160, :, 3] = bad
        leaves = [t.detach().requires_grad_() for t in broken[:3]]
        out = ops.attention(*leaves, q_docs=ids, k_docs=ids, causal=causal)
        grads = torch.autograd.grad(out, leaves, broken[3])
        assert torch.equal(out[:, :90], clean[0][:, :90]) and torch.equal(out[:, 160:], clean[0][:, 160:])
        for got, want in zip((out, *grads), (clean[0], *clean[1])):
            # f16's dS has another power of two as its scale without the broken
            # recording: the smallest of them round otherwise
            for part in (slice(0, 90), slice(160, T)):
                room = 2 * ref.U[dtype] * want[:, part].abs().max()
                assert ((got[:, part] - want[:, part]).abs() <= room).all()
            assert not torch.isfinite(got[:, 90:160]).all()
    # causal: what comes after a query, in few-query form and in tiles
    for Tq in (T, 3):
        k2, v2 = k.clone(), v.clone()
        k2[:, 150:], v2[:, 150:] = bad, bad
        out = ops.attention(q[:, :Tq], k2, v2, causal=True, q_start=149 - (Tq - 1) if Tq < T else 0)
        want = ops.attention(q[:, :Tq], k, v, causal=True, q_start=149 - (Tq - 1) if Tq < T else 0)
        n = 150 if Tq == T else Tq
        assert torch.equal(out[:, :n], want[:, :n])
        assert torch.isnan(out[:, n:]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_layouts(ops, dtype):
    g = gen(11)
    B, T, H, D = 2, 150, 4, 64
    qkv = randn(g, B, T, 3 * H, D, dtype=dtype)
    heads_first = randn(g, B, H, T, D, dtype=dtype).transpose(1, 2)
    token_first = randn(g, T, B, H, D, dtype=dtype).transpose(0, 1)
    odd = randn(g, B, T, H, D + 3, dtype=dtype)[..., 3:]  # rows that start off 16-byte boundaries
    far = randn(g, B, T, H, 2 * D, dtype=dtype)[..., ::2]  # elements apart
    shared = randn(g, 1, T, H, D, dtype=dtype).expand(B, T, H, D)
    dy = randn(g, B, H, T, D, dtype=dtype).transpose(1, 2)
    for q, k, v in ((qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]), (heads_first, token_first, heads_first),
                    (token_first, odd, qkv[:, :, :H]), (odd, far, odd), (far, shared, shared)):
        check_attention(ops, q, k, v, f"{q.stride()} {k.stride()}", dy=dy)
    q = qkv[:, :, :H]
    out = ops.attention(q.detach().requires_grad_(), q, q)
    (d,) = torch.autograd.grad(out.sum(), [out.grad_fn.next_functions[0][0].variable])
    assert torch.isfinite(d).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [40, 64])
def test_attention_empty(ops, dtype, dim):
    for B, Tq, Tk in ((0, 5, 5), (2, 0, 5), (2, 5, 0)):
        q, k, v, dy, g = make((B, Tq, Tk, 2, 1, dim), dtype)
        table = randn(g, 32, 2, dtype=dtype)
        out, grads = check_attention(ops, q, k, v, f"{B} {Tq} {Tk}", dy=dy, table=table)
        assert all(torch.equal(d, torch.zeros_like(d)) for d in grads)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_rows_and_starts(ops, dtype):
    # queries before, inside and after the keys; causal rows that see nothing
    q, k, v, dy, g = make((3, 140, 200, 2, 1, 64), dtype)
    table = randn(g, 32, 2, dtype=dtype)
    starts = lengths(-100, 30, 500)
    out, _ = check_attention(ops, q, k, v, "starts", dy=dy, causal=True, q_start=starts, table=table)
    assert torch.equal(out[0, :100], torch.zeros_like(out[0, :100]))
    check_attention(ops, q, k, v, "one-sided", dy=dy, table=table, bidirectional=False, max_distance=70)
    check_attention(ops, q, k, v, "prefix", dy=dy, causal=True, prefix=lengths(0, 250, 100), k_lens=lengths(200, 90, 1))


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_large_scores(ops, dtype):
    q, k, v, dy, g = make((1, 150, 300, 2, 2, 64), dtype)
    check_attention(ops, q * 20, k * 20, v, "large scores", dy=dy)
    check_attention(ops, q * 20, k * 20, v, "large scores, capped", dy=dy, softcap=30.0)
    # a single key takes all: weights of 1 and 0, a running maximum that rises in every tile
    k2 = k * torch.linspace(0.1, 30, 300, device="cuda").to(dtype)[None, :, None, None]
    check_attention(ops, q * 4, k2, v, "rising", dy=dy)


@pytest.mark.parametrize("dtype", [F32, F16])
def test_attention_differences(ops, dtype):
    g = gen(13)
    q, k, v, dy, _ = make((1, 40, 60, 4, 2, 64), dtype)
    table = randn(g, 16, 4, dtype=dtype)
    kw = {"causal": True, "softcap": 8.0, "max_distance": 40}
    out, grads = check_attention(ops, q, k, v, "differences", dy=dy, table=table, **kw)
    tensors = [q, k, v, table]
    want = ref.attention(q, k, v, dy=dy, table=table, **kw)
    for n, name in enumerate(("dq", "dk", "dv", "dtable")):
        step = randn(g, *tensors[n].shape).double()

        def loss(s):
            # the definition on inputs moved by s, in 64 bits
            moved = [t.double() for t in tensors]
            moved[n] = moved[n] + s * step
            Q, K, V, Tb = moved
            K, V = K.repeat_interleave(2, 2), V.repeat_interleave(2, 2)
            z = torch.einsum("bihd,bjhd->bhij", Q, K) / 8.0
            z = 8.0 * torch.tanh(z / 8.0)
            o = torch.arange(60)[None, :] - (20 + torch.arange(40))[:, None]
            known = ref.bucket_tensor(-60, 60, 16, 40, True)
            z = z + Tb[known[o + 60].cuda()].permute(2, 0, 1)
            z = z.masked_fill((o > 0).cuda(), -math.inf)
            return float((torch.einsum("bhij,bjhd->bihd", torch.softmax(z, -1), V) * dy.double()).sum())

        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = float((grads[n].double() * step).sum())
        room = float((want[name][1].to(step.device) * step.abs()).sum())
        assert abs(got - slope) <= room + 1e-6 * abs(slope) + 1e-6, name


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_same_bits_and_streams(ops, dtype):
    q, k, v, dy, g = make((2, 300, 300, 4, 2, 64), dtype)
    table = randn(g, 32, 4, dtype=dtype)

    def once():
        leaves = [t.detach().requires_grad_() for t in (q, k, v, table)]
        out = ops.attention(*leaves[:3], table=leaves[3], causal=True)
        return [out.detach(), *torch.autograd.grad(out, leaves, dy)]

    first = once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = once()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_attention_graph(ops):
    # recorded once, replayed on new values
    q, k, v, _, g = make((2, 1, 300, 8, 2, 64), BF16)
    table = randn(g, 32, 8, dtype=BF16)
    lens = lengths(300, 120)
    ops.attention(q, k, v, table=table, k_lens=lens)  # makes the bucket map
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.attention(q, k, v, table=table, k_lens=lens)
    for seed in (1, 2):
        q.copy_(randn(gen(seed), *q.shape, dtype=BF16))
        lens.copy_(lengths(7, 299))
        graph.replay()
        ref.close(out, *ref.attention(q, k, v, table=table, k_lens=lens)["out"], "replayed")


def test_training_graph(ops):
    # a training step recorded once, replayed on new values
    q, k, v, dy, g = make((2, 200, 200, 4, 2, 64), BF16)
    table = randn(g, 32, 4, dtype=BF16)
    w = randn(g, 64, dtype=BF16)
    leaves = [t.requires_grad_() for t in (q, k, v, table, w)]
    ids = docs_of(200, [(0, 120), (1, 70)], [(3, 200)])

    def step():
        out = ops.attention(ops.layer_norm(q, w), k, v, table=table, causal=True, q_docs=ids, k_docs=ids)
        return [out.detach(), *torch.autograd.grad(out, leaves, dy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        with torch.no_grad():
            for t in (q, k, v):
                t.copy_(randn(gen(seed), *t.shape, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(replayed, step()))


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_on_new_threads(ops, dtype):
    # a thread whose first CUDA work is the operator, its memory from the cache
    import threading

    q, k, v, dy, g = make((2, 300, 300, 4, 2, 64), dtype)
    got = {}

    def once(name):
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        out = ops.attention(*leaves, causal=True)
        got[name] = [out.detach(), *torch.autograd.grad(out, leaves, dy)]

    once("here")
    again = got.pop("here")
    torch.cuda.synchronize()
    for n in range(3):
        t = threading.Thread(target=once, args=(n,))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, got.pop(n)))


# ---------------------------------------------------------------------------
# refusals

def test_refusals(ops):
    x = torch.randn(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    for call, error in [
        (lambda: ops.layer_norm(x.cpu()), ValueError),
        (lambda: ops.layer_norm(x.double()), TypeError),
        (lambda: ops.layer_norm(x, w[:7]), ValueError),
        (lambda: ops.layer_norm(x, w.half()), TypeError),
        (lambda: ops.layer_norm(x.half(), w.half(), w), TypeError),
        (lambda: ops.layer_norm(x, w, eps=-1.0), ValueError),
        (lambda: ops.layer_norm(x[:, :0]), ValueError),
        (lambda: ops.layer_norm(x, w.cpu()), ValueError),
        (lambda: ops.relative_bias(x[0], 3, 3), ValueError),
        (lambda: ops.relative_bias(x.long(), 3, 3), TypeError),
        (lambda: ops.relative_bias(x, -1, 3), ValueError),
        (lambda: ops.relative_bias(x, 3, 3, max_distance=4096), ValueError),
        (lambda: ops.relative_bias(x, 3, 3, max_distance=1), ValueError),
        (lambda: ops.relative_bias(x[:3], 3, 3), ValueError),
    ]:
        with pytest.raises(error):
            call()
    q = torch.randn(2, 5, 4, 16, device="cuda")
    k = torch.randn(2, 7, 2, 16, device="cuda")
    ids = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    for kw, error in [
        ({"k": k.half()}, TypeError), ({"k": k.cpu()}, ValueError), ({"v": k[:, :6]}, ValueError),
        ({"q": q[:, :, :3]}, ValueError), ({"q": q[..., :8]}, ValueError), ({"q": q[:1]}, ValueError),
        ({"softcap": -1.0}, ValueError), ({"scale": math.inf}, ValueError),
        ({"prefix": lengths(1, 1)}, ValueError), ({"k_lens": lengths(1)}, ValueError),
        ({"k_lens": lengths(1, 1).long()}, TypeError), ({"q_docs": ids}, ValueError),
        ({"q_docs": ids, "k_docs": ids}, ValueError), ({"table": torch.randn(32, 2, device="cuda")}, ValueError),
        ({"table": torch.randn(32, 4, device="cuda").half()}, TypeError),
        ({"slopes": torch.ones(2, device="cuda")}, ValueError),
        ({"slopes": torch.ones(4, device="cuda", requires_grad=True)}, RuntimeError),
        ({"q": q.double(), "k": k.double(), "v": k.double()}, TypeError),
        ({"q_start": lengths(1)}, ValueError),
    ]:
        args = {"q": q, "k": k, "v": kw.get("k", k), **kw}
        with pytest.raises(error):
            ops.attention(args.pop("q"), args.pop("k"), args.pop("v"), **args)
    big = torch.zeros(1, 2, 1, 257, device="cuda")
    with pytest.raises(ValueError):
        ops.attention(big, big, big)
    # once differentiable, and still usable after a refusal
    xg = x.clone().requires_grad_()
    (d,) = torch.autograd.grad(ops.layer_norm(xg).square().sum(), xg, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(d.sum(), xg)


def test_no_kernel_gave_up(ops):
    from mel_spectrogram_gb300 import FM_OK

    assert ops.poll_error() == FM_OK
