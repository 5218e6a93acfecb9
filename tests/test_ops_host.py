"""Host-only tests of the frame-encoder operators' C ABI: what the header
declares, the argument structs, and refusals that need no GPU."""
from __future__ import annotations

import ctypes as C
import os
import re

import pytest

from mel_spectrogram_gb300 import _binding as fb

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fm_ops.h")


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300.build import build

    build()
    from mel_spectrogram_gb300 import ops

    return ops


def header() -> str:
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_and_binding_agree(ops):
    assert sorted(set(re.findall(r"\b(fm_[a-z_0-9]+)\s*\(", header()))) == sorted(ops.EXPORTS)
    L = ops._lib()
    for name in ops.EXPORTS:
        getattr(L, name)


@pytest.mark.parametrize("struct,packer", [("fm_layer_norm_args", "_NORM"), ("fm_relative_bias_args", "_BIAS"),
                                           ("fm_attention_args", "_ATTN")])
def test_structs_match_their_packers(ops, struct, packer):
    body = next(b for b, n in re.findall(r"typedef struct \{(.*?)\}\s*(\w+);", header(), flags=re.S) if n == struct)
    codes = ""
    for line in body.split(";"):
        line = " ".join(line.split())
        if not line:
            continue
        base = re.match(r"(const )?(\w+)", line).group(2)
        for name in line.split(","):
            count = int(re.search(r"\[(\d+)\]", name).group(1)) if "[" in name else 1
            # a pointer's star stands with its own name, or with the type of the first
            star = "*" in name
            codes += ("Q" if star else {"int64_t": "q", "double": "d"}[base]) * count
    fmt = getattr(ops, packer).format.lstrip("=")
    assert "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([qdQ])", fmt)) == codes


def norm_args(ops, **kw):
    a = dict(rows=4, width=8, dtype=fb.FM_F32, ptype=fb.FM_F32, xs=8, ys=8, eps=1e-5, x=64, y=64) | kw
    return ops._NORM.pack(a["rows"], a["width"], a["dtype"], a["ptype"], a["xs"], a["ys"], 8, 8, a["eps"], a["x"], 0,
                          0, a["y"], 0, 0, 0, 0, 0, 0, 0, 0)


def test_norm_refusals(ops):
    L = ops._lib()
    for kw in (dict(rows=-1), dict(width=0), dict(width=1 << 25), dict(dtype=fb.FM_I16), dict(ptype=fb.FM_F16),
               dict(xs=7), dict(ys=-8), dict(eps=-1.0), dict(eps=float("nan")), dict(x=0), dict(y=0)):
        assert L.fm_layer_norm_forward(norm_args(ops, **kw), None) == fb.FM_ERR_INVALID_ARG, kw
    assert L.fm_layer_norm_forward(norm_args(ops, rows=0, x=0, y=0), None) == fb.FM_OK
    assert L.fm_layer_norm_backward(norm_args(ops), None) == fb.FM_ERR_INVALID_ARG
    assert L.fm_layer_norm_workspace(norm_args(ops, width=0)) == -1
    assert L.fm_layer_norm_workspace(norm_args(ops)) >= 2 * 8 * 4
    for f in (L.fm_layer_norm_forward, L.fm_relative_bias_forward, L.fm_attention_forward, L.fm_layer_norm_backward,
              L.fm_relative_bias_backward, L.fm_attention_backward):
        assert f(None, None) == fb.FM_ERR_INVALID_ARG


def test_bucket_refusals(ops):
    L = ops._lib()
    h = C.c_void_p(1)
    for nb, far, both in ((3, 100, 1), (2, 100, 1), (1, 100, 0), (4098, 2048, 1), (32, 8, 1), (32, 2049, 1),
                          (32, 16, 0), (32, -5, 1)):
        assert L.fm_buckets_create(C.byref(h), nb, far, both) == fb.FM_ERR_INVALID_ARG, (nb, far, both)
        assert h.value is None
    assert L.fm_buckets_create(None, 32, 128, 1) == fb.FM_ERR_INVALID_ARG
    assert L.fm_buckets_map(None, None) == fb.FM_ERR_INVALID_ARG
    assert L.fm_buckets_destroy(None) == fb.FM_OK


def attn_args(ops, **kw):
    a = dict(batch=2, q_len=3, k_len=5, heads=4, kv_heads=2, dim=64, dtype=fb.FM_BF16, scale=0.125, cap=0.0, q=64,
             k=64, v=64, out=64, q_docs=0, k_docs=0, handle=0, table=0, ttype=0) | kw
    return ops._ATTN.pack(a["batch"], a["q_len"], a["k_len"], a["heads"], a["kv_heads"], a["dim"], a["dtype"], 0,
                          a["scale"], a["cap"], a["q"], a["k"], a["v"], a["out"], *([0] * 12), 0, a["q_docs"],
                          a["k_docs"], 0, 0, 0, ops.Q_START_END, a["handle"], a["table"], a["ttype"], 0, 0, 0, 0, 0,
                          *([0] * 12), 0, 0, 0)


def test_attention_refusals(ops):
    L = ops._lib()
    inf, nan = float("inf"), float("nan")
    for kw in (dict(batch=-1), dict(batch=65536), dict(q_len=-1), dict(k_len=1 << 29), dict(heads=0), dict(kv_heads=0),
               dict(kv_heads=3), dict(dim=0), dict(dtype=fb.FM_I16), dict(dtype=9), dict(scale=inf), dict(scale=nan),
               dict(cap=-1.0), dict(cap=nan), dict(q_docs=64), dict(k_docs=64), dict(q=0), dict(out=0), dict(k=0),
               dict(v=0)):
        assert L.fm_attention_forward(attn_args(ops, **kw), None) == fb.FM_ERR_INVALID_ARG, kw
    assert L.fm_attention_forward(attn_args(ops, dim=257), None) == fb.FM_ERR_UNSUPPORTED
    assert L.fm_attention_workspace(attn_args(ops, dim=257), 1) == -1
    assert L.fm_attention_workspace(attn_args(ops), 1) > 0
    for kw in (dict(batch=0), dict(q_len=0)):
        assert L.fm_attention_forward(attn_args(ops, q=0, out=0, **kw), None) == fb.FM_OK
    # a backward call without its workspace, or without the tensors it reads
    assert L.fm_attention_backward(attn_args(ops), None) == fb.FM_ERR_INVALID_ARG


def test_functions_refuse_host_tensors(ops):
    x = torch.randn(2, 3, 4, 8)
    with pytest.raises(ValueError):
        ops.layer_norm(x)
    with pytest.raises(ValueError):
        ops.relative_bias(x[0, 0], 3, 3)
    with pytest.raises(ValueError):
        ops.attention(x, x, x)
    with pytest.raises(ValueError):
        ops.bucket_map(32, device="cpu")
