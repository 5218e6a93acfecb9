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
    L = ops.library()
    for name in ops.EXPORTS:
        getattr(L, name)


def struct_of(name: str):
    """A ctypes structure from the header's text."""
    body = next(b for b, n in re.findall(r"typedef struct \{(.*?)\}\s*(\w+);", header(), flags=re.S) if n == name)
    fields = []
    for line in body.split(";"):
        line = " ".join(line.split())
        if not line:
            continue
        base = re.match(r"(?:const )?(\w+)", line).group(1)
        for part in line.split(","):
            field = re.search(r"(\w+)(?:\[(\d+)\])?$", part.strip())
            kind = C.c_void_p if "*" in part else {"int64_t": C.c_int64, "double": C.c_double}[base]
            fields.append((field.group(1), kind * int(field.group(2)) if field.group(2) else kind))
    return type(name, (C.Structure,), {"_fields_": fields})


def args_of(name: str, **values):
    a = struct_of(name)()
    for k, v in values.items():
        setattr(a, k, v)
    return C.byref(a)


def test_structs_have_the_compilers_size():
    import subprocess
    import tempfile

    names = ["fm_layer_norm_args", "fm_relative_bias_args", "fm_attention_args"]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "s.c"), os.path.join(d, "s")
        with open(src, "w") as f:
            f.write('#include <stdio.h>\n#include "fm_ops.h"\nint main(void) {\n')
            f.writelines(f'  printf("%zu\\n", sizeof({n}));\n' for n in names)
            f.write("  return 0;\n}\n")
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        sizes = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert sizes == [C.sizeof(struct_of(n)) for n in names]


def norm_args(**kw):
    a = dict(rows=4, width=8, dtype=fb.FM_F32, param_dtype=fb.FM_F32, x_stride=8, y_stride=8, dy_stride=8,
             dx_stride=8, eps=1e-5, x=64, y=64)
    return args_of("fm_layer_norm_args", **(a | kw))


def test_norm_refusals(ops):
    L = ops.library()
    for kw in (dict(rows=-1), dict(width=0), dict(width=1 << 25), dict(dtype=fb.FM_I16), dict(param_dtype=fb.FM_F16),
               dict(x_stride=7), dict(y_stride=-8), dict(eps=-1.0), dict(eps=float("nan")), dict(x=0), dict(y=0)):
        assert L.fm_layer_norm_forward(norm_args(**kw), None) == fb.FM_ERR_INVALID_ARG, kw
    assert L.fm_layer_norm_forward(norm_args(rows=0, x=0, y=0), None) == fb.FM_OK
    assert L.fm_layer_norm_backward(norm_args(), None) == fb.FM_ERR_INVALID_ARG
    assert L.fm_layer_norm_workspace(norm_args(width=0)) == -1
    assert L.fm_layer_norm_workspace(norm_args()) >= 2 * 8 * 4
    for f in (L.fm_layer_norm_forward, L.fm_relative_bias_forward, L.fm_attention_forward, L.fm_layer_norm_backward,
              L.fm_relative_bias_backward, L.fm_attention_backward):
        assert f(None, None) == fb.FM_ERR_INVALID_ARG


def test_bucket_refusals(ops):
    L = ops.library()
    h = C.c_void_p(1)
    for nb, far, both in ((3, 100, 1), (2, 100, 1), (1, 100, 0), (4098, 2048, 1), (32, 8, 1), (32, 2049, 1),
                          (32, 16, 0), (32, -5, 1)):
        assert L.fm_buckets_create(C.byref(h), nb, far, both) == fb.FM_ERR_INVALID_ARG, (nb, far, both)
        assert h.value is None
    assert L.fm_buckets_create(None, 32, 128, 1) == fb.FM_ERR_INVALID_ARG
    assert L.fm_buckets_map(None, None) == fb.FM_ERR_INVALID_ARG
    assert L.fm_buckets_destroy(None) == fb.FM_OK


def attn_args(**kw):
    a = dict(batch=2, q_len=3, k_len=5, heads=4, kv_heads=2, dim=64, dtype=fb.FM_BF16, scale=0.125, softcap=0.0, q=64,
             k=64, v=64, out=64, q_start_all=-(1 << 63))
    return args_of("fm_attention_args", **(a | kw))


def test_attention_refusals(ops):
    L = ops.library()
    inf, nan = float("inf"), float("nan")
    for kw in (dict(batch=-1), dict(batch=65536), dict(q_len=-1), dict(k_len=1 << 29), dict(heads=0), dict(kv_heads=0),
               dict(kv_heads=3), dict(dim=0), dict(dtype=fb.FM_I16), dict(dtype=9), dict(scale=inf), dict(scale=nan),
               dict(softcap=-1.0), dict(softcap=nan), dict(q_docs=64), dict(k_docs=64), dict(q=0), dict(out=0),
               dict(k=0), dict(v=0)):
        assert L.fm_attention_forward(attn_args(**kw), None) == fb.FM_ERR_INVALID_ARG, kw
    assert L.fm_attention_forward(attn_args(dim=257), None) == fb.FM_ERR_UNSUPPORTED
    assert L.fm_attention_workspace(attn_args(dim=257), 1) == -1
    assert L.fm_attention_workspace(attn_args(), 1) > 0
    for kw in (dict(batch=0), dict(q_len=0)):
        assert L.fm_attention_forward(attn_args(q=0, out=0, **kw), None) == fb.FM_OK
    # a backward call without its workspace, or without the tensors it reads
    assert L.fm_attention_backward(attn_args(), None) == fb.FM_ERR_INVALID_ARG


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
