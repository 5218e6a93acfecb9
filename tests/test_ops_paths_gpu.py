"""The frame-encoder operators on the paths that only long, split or far-reaching
calls take: keys split over blocks in tiles and for few queries with either
join, documents for few queries, biases that reach 2048 places, offsets past 32
bits."""
from __future__ import annotations

import math

import pytest
import torch

from tests import ops_reference as ref
from tests import test_ops_gpu as base

pytestmark = pytest.mark.gpu

F32, F16, BF16 = base.F32, base.F16, base.BF16
TYPES = base.TYPES


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300 import ops

    return ops


# ---------------------------------------------------------------------------
# few blocks and many keys: the tiled forward pass splits them

SPLIT = {
    "plain": lambda s, t, g: {},
    "causal": lambda s, t, g: {"causal": True},
    "starts": lambda s, t, g: {"causal": True, "q_start": torch.full((s[0],), 500, dtype=torch.int32, device="cuda")},
    "all": lambda s, t, g: {"causal": True, "softcap": 10.0, "table": base.randn(g, 32, s[3]), "max_distance": 100,
                            "prefix": torch.full((s[0],), 20, dtype=torch.int32, device="cuda"),
                            "k_lens": torch.full((s[0],), s[2] - 131, dtype=torch.int32, device="cuda")},
    "short": lambda s, t, g: {"k_lens": torch.full((s[0],), 300, dtype=torch.int32, device="cuda")},
    "slopes": lambda s, t, g: {"slopes": torch.rand(s[3], device="cuda", generator=g) * 0.1},
}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128, 72])
@pytest.mark.parametrize("option", list(SPLIT))
def test_split_tiles(ops, option, dim, dtype):
    for shape in ((1, 40, 1500, 2, 1, dim), (2, 300, 1025, 2, 2, dim)):
        q, k, v, dy, g = base.make(shape, dtype)
        kw = SPLIT[option](shape, dtype, g)
        base.check_attention(ops, q, k, v, f"{shape} {option} {dtype}", **kw)
        base.check_attention(ops, q, k, v, f"{shape} {option} {dtype}", dy=dy, **kw)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_split_tiles_documents(ops, dim, dtype):
    q, k, v, dy, g = base.make((1, 1300, 1300, 2, 1, dim), dtype)
    ids = base.docs_of(1300, [(4, 500), (-1, 60), (2, 333), (9, 300)])
    table = base.randn(g, 32, 2, dtype=dtype)
    q, dy, q_ids = q[:, 450:750], dy[:, 450:750], ids[:, 450:750].contiguous()
    for causal in (False, True):
        clean = base.check_attention(ops, q, k, v, "split documents", dy=dy, q_docs=q_ids, k_docs=ids, causal=causal,
                                     q_start=450, table=table)[0]
        # a broken recording beside it, through the second launch of the splits
        k2, v2 = k.clone(), v.clone()
        k2[:, 560:893], v2[:, 560:893] = math.inf, math.nan
        out = ops.attention(q, k2, v2, q_docs=q_ids, k_docs=ids, causal=causal, q_start=450, table=table)
        assert torch.equal(out[:, :50], clean[:, :50]) and out[:, 110:].isnan().all()
        assert torch.equal(out[:, 50:110], torch.zeros_like(out[:, 50:110]))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_splits(ops, dim, dtype):
    # from 64 splits on the join takes 32 warps: 33000 keys in tiles, 20000 for few queries
    q, k, v, _, _ = base.make((1, 40, 33000, 1, 1, dim), dtype)
    base.check_attention(ops, q, k, v, "40 x 33000")
    base.check_attention(ops, q, k, v, "40 x 33000", causal=True, k_lens=base.lengths(30001))
    for heads, kv_heads, Tq in ((2, 1, 1), (4, 2, 5)):
        q, k, v, _, g = base.make((1, Tq, 20000, heads, kv_heads, dim), dtype)
        table = base.randn(g, 32, heads, dtype=dtype)
        base.check_attention(ops, q, k, v, f"{Tq} x 20000", causal=True, table=table)
        base.check_attention(ops, q, k, v, f"{Tq} x 20000", k_lens=base.lengths(17), table=table)
        base.check_attention(ops, q, k, v, f"{Tq} x 20000", k_lens=base.lengths(0))


# ---------------------------------------------------------------------------
# documents for few queries

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("Tq", [1, 5, 16, 30])
def test_few_queries_documents(ops, Tq, dim, dtype):
    B, Tk = 3, 700
    q, k, v, dy, g = base.make((B, Tq, Tk, 8, 2, dim), dtype)
    k_ids = base.docs_of(Tk, [(0, 300), (1, 400)], [(3, 20), (-1, 100), (3, 300)], [(7, 700)])
    q_ids = torch.randint(-1, 4, (B, Tq), dtype=torch.int32, device="cuda", generator=g)
    q_ids[2] = 6  # meets nothing
    table = base.randn(g, 32, 8, dtype=dtype)
    for kw in ({}, {"causal": True}, {"k_lens": base.lengths(650, 333, 1), "softcap": 20.0}, {"table": table}):
        out = base.check_attention(ops, q, k, v, f"{kw.keys()}", q_docs=q_ids, k_docs=k_ids, **kw)
        assert torch.equal(out[2], torch.zeros_like(out[2]))
        base.check_attention(ops, q, k, v, f"{kw.keys()}", dy=dy, q_docs=q_ids, k_docs=k_ids, **kw)


# ---------------------------------------------------------------------------
# biases that reach 2048 places

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("both", [True, False])
def test_far_bias(ops, both, dim, dtype):
    for shape, kw in (((1, 400, 2600, 2, 1, dim), {"q_start": 2100}), ((1, 2500, 200, 1, 1, dim), {"q_start": 0}),
                      ((1, 300, 300, 2, 2, dim), {"q_start": -2000}), ((1, 3, 2600, 2, 1, dim), {"causal": True})):
        q, k, v, dy, g = base.make(shape, dtype)
        table = base.randn(g, 64, shape[3], dtype=dtype)
        base.check_attention(ops, q, k, v, f"{shape} {both}", dy=dy, table=table, max_distance=2048, bidirectional=both, **kw)


# ---------------------------------------------------------------------------
# offsets past 32 bits

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_offsets(ops, dtype):
    # rows of the batch, then the first and the last token, more than 2^31 elements apart
    for Tq, Tk in ((1, 130), (70, 130)):
        B, H, D = 2, 2, 64
        q, k, v, dy, _ = base.make((B, Tq, Tk, H, H, D), dtype)
        space = torch.empty(Tk * 2 ** 24, dtype=dtype, device="cuda")
        by_row = space.as_strided((B, Tk, H, D), (2 ** 31 + 4096, H * D, D, 1))
        by_row.copy_(k)
        base.check_attention(ops, q, by_row, v, "rows apart", dy=dy)
        base.check_attention(ops, q, k, by_row, "rows apart", dy=dy)
        by_token = space.as_strided((1, Tk, H, D), (Tk * 2 ** 24, 2 ** 24, D, 1))
        by_token.copy_(v[:1])
        base.check_attention(ops, q[:1], by_token, v[:1], "tokens apart", dy=dy[:1])
        base.check_attention(ops, q[:1], k[:1], by_token, "tokens apart", dy=dy[:1])
        del space, by_row, by_token
        torch.cuda.empty_cache()


def test_norm_offsets(ops):
    g = base.gen(1)
    rows, width = 2 ** 21 + 5, 1024
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    x[-9:] = base.randn(g, 9, width, dtype=BF16)
    dy = torch.zeros_like(x)
    dy[-9:] = base.randn(g, 9, width, dtype=BF16)
    w, b = base.randn(g, width, dtype=BF16), base.randn(g, width, dtype=BF16)
    y, (dx, dw, db) = base.run_norm(ops, x, w, b, 1e-5, dy)
    want = ref.norm(x[-9:], w, b, 1e-5, dy[-9:])
    for name, got in (("out", y[-9:]), ("dx", dx[-9:]), ("dweight", dw), ("dbias", db)):
        ref.close(got, *want[name], name)
    assert torch.equal(y[:-9], b.expand(rows - 9, width)) and not dx[:-9].any()
    del x, dy, y, dx
    torch.cuda.empty_cache()


def test_relative_bias_offsets(ops):
    g = base.gen(2)
    H, Tq, Tk = 16, 11000, 12300
    table = base.randn(g, 32, H, dtype=BF16).requires_grad_()
    out = ops.relative_bias(table, Tq, Tk)
    dy = torch.zeros(H, Tq, Tk, dtype=BF16, device="cuda")
    dy[-1, -40:] = base.randn(g, 40, Tk, dtype=BF16)
    (d,) = torch.autograd.grad(out, table, dy)
    want = ref.dense_bias(table.detach()[:, -1:], 40, Tk, Tk - 40, 128, True, dy[-1:, -40:])
    ref.close(out[-1:, -40:], *want["out"], "last rows")
    ref.close(d[:, -1:], *want["dtable"], "last head")
    assert not d[:, :-1].any()
    first = ref.dense_bias(table.detach(), 3, Tk, Tk - Tq, 128, True)
    ref.close(out[:, :3], *first["out"], "first rows")
    del out, dy
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# both sides of every limit between the kernels for few queries and in tiles

@pytest.mark.parametrize("dim", [64, 72, 128])
@pytest.mark.parametrize("Tq", [16, 17, 32, 33])
def test_choice_of_kernel(ops, Tq, dim):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # batch entries of heads 4 (2 and 4 of them sharing keys) around half and all of the SMs' blocks
    for kv_heads in (2, 1):
        for batch in {sms // 8, sms // 8 + 1, sms // 4, sms // 4 + 1}:
            q, k, v, _, _ = base.make((batch, Tq, 150, 4, kv_heads, dim), BF16)
            base.check_attention(ops, q, k, v, f"{batch} {Tq} {kv_heads} {dim}", causal=True)
