"""Operators of a model over mel frames (include/fm_ops.h): layer norm, a
learned position bias by distance buckets, and attention over frames.

Functions on CUDA tensors with autograd support. Every computation runs in the
library's own kernels; this module checks arguments, allocates outputs and
workspaces and passes pointers, on the current stream of the tensors' device.

    y = layer_norm(x, weight, bias)                      # (..., width)
    b = relative_bias(table, q_len, k_len)               # (heads, q_len, k_len)
    o = attention(q, k, v, table=table, q_docs=d, k_docs=d)   # (batch, len, heads, dim)
"""
from __future__ import annotations

import ctypes as C
import math
import struct

import torch

from . import _binding as fb

# every symbol include/fm_ops.h declares
EXPORTS = [
    "fm_layer_norm_forward",
    "fm_layer_norm_backward",
    "fm_layer_norm_workspace",
    "fm_buckets_create",
    "fm_buckets_map",
    "fm_buckets_destroy",
    "fm_relative_bias_forward",
    "fm_relative_bias_backward",
    "fm_relative_bias_workspace",
    "fm_attention_forward",
    "fm_attention_backward",
    "fm_attention_workspace",
    "fm_ops_poll_error",
]

_TYPES = {torch.float32: fb.FM_F32, torch.float16: fb.FM_F16, torch.bfloat16: fb.FM_BF16}
Q_START_END = -(1 << 63)

# the argument structs of fm_ops.h, field by field (every field has 8 bytes)
_NORM = struct.Struct("=8qd3Q" + "Q" + "2Q" + "Q3Q" + "Qq")
_BIAS = struct.Struct("=5q" + "6Q" + "q")
_ATTN = struct.Struct("=8q2d" + "4Q" + "12q" + "Q" + "5Q" + "q" + "2Qq" + "Q" + "Q3Q" + "12q" + "Q" + "Qq")

_bound = None


def _lib():
    """The library with the prototypes of fm_ops.h (always the release build:
    the debug build holds the mel kernels only)."""
    global _bound
    if _bound is None:
        L = fb.load(fb.LIB_PATH)
        vp, ci = C.c_void_p, C.c_int
        for op in ("layer_norm", "relative_bias", "attention"):
            for way in ("forward", "backward"):
                f = getattr(L, f"fm_{op}_{way}")
                f.argtypes, f.restype = [C.c_char_p, vp], ci
            f = getattr(L, f"fm_{op}_workspace")
            f.argtypes, f.restype = [C.c_char_p] + ([ci] if op == "attention" else []), C.c_int64
        L.fm_buckets_create.argtypes, L.fm_buckets_create.restype = [C.POINTER(vp), ci, ci, ci], ci
        L.fm_buckets_map.argtypes, L.fm_buckets_map.restype = [vp, vp], ci
        L.fm_buckets_destroy.argtypes, L.fm_buckets_destroy.restype = [vp], ci
        L.fm_ops_poll_error.argtypes, L.fm_ops_poll_error.restype = [], ci
        _bound = L
    return _bound


def _call(name: str, args: bytes, device: torch.device) -> None:
    f = getattr(_lib(), name)
    stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        status = f(args, stream)
    else:
        with torch.cuda.device(device):
            status = f(args, stream)
    if status:
        raise fb.FmError(status, name)


def _need_cuda(**tensors) -> torch.device:
    device = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the operators run only on the GPU)")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other inputs on {device}")
    return device


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _wants_grad(*tensors) -> bool:
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


# ---------------------------------------------------------------------------
# layer norm

def _rows(t: torch.Tensor, width: int):
    """t as (2-D tensor with adjacent elements in a row, its row stride); a
    view where the strides allow one, a copy otherwise."""
    if not t.is_contiguous():
        t = t.reshape(-1, width)
        if t.stride(1) != 1 and width > 1:
            t = t.contiguous()
        if t.shape[0] > 1 and t.stride(0) < width:
            t = t.contiguous()
        return t, max(t.stride(0), width)
    return t, width


def _norm_forward(x, weight, bias, eps, stats: bool):
    width = x.shape[-1]
    rows = x.numel() // width
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    x2, stride = _rows(x, width)
    mean = rstd = None
    if stats:
        mean, rstd = torch.empty(2, rows, dtype=torch.float32, device=x.device)
    ptype = weight if weight is not None else bias
    args = _NORM.pack(rows, width, _TYPES[x.dtype], _TYPES[x.dtype if ptype is None else ptype.dtype], stride, width,
                      0, 0, eps, x2.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd), 0, 0,
                      0, 0, 0, 0)
    _call("fm_layer_norm_forward", args, x.device)
    return y, mean, rstd


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _norm_forward(x, weight, bias, eps, True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.eps = eps
        ctx.params = (None if weight is None else weight.dtype, None if bias is None else bias.dtype)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        width, device = x.shape[-1], x.device
        rows = x.numel() // width
        need = ctx.needs_input_grad
        x2, xs = _rows(x, width)
        dy2, dys = _rows(dy, width)
        dx = torch.empty(x.shape, dtype=x.dtype, device=device) if need[0] else None
        ptype = ctx.params[0] or ctx.params[1] or x.dtype
        dw = torch.empty(width, dtype=ptype, device=device) if need[1] else None
        db = torch.empty(width, dtype=ptype, device=device) if need[2] else None

        def pack(work, size):
            return _NORM.pack(rows, width, _TYPES[x.dtype], _TYPES[ptype], xs, 0, dys, width, ctx.eps, x2.data_ptr(),
                              _ptr(weight), 0, 0, mean.data_ptr(), rstd.data_ptr(), dy2.data_ptr(), _ptr(dx),
                              _ptr(dw), _ptr(db), work, size)

        work, size = None, 0
        if dw is not None or db is not None:
            size = _lib().fm_layer_norm_workspace(pack(0, 0))
            work = torch.empty(size, dtype=torch.uint8, device=device)
        _call("fm_layer_norm_backward", pack(_ptr(work), size), device)
        return dx, dw, db, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of x over its last dimension, in x's type.

    x: (..., width) float32, float16 or bfloat16, any strides (rows whose
    elements are not adjacent are copied first). weight, bias: (width,), of
    x's type or float32 (both the same type), or None for ones and zeros.
    Statistics are 32-bit: the mean, then the mean squared deviation from it.
    Differentiable in x, weight and bias (once).
    """
    device = _need_cuda(x=x, weight=weight, bias=bias)
    if x.dtype not in _TYPES:
        raise TypeError(f"x: dtype {x.dtype} not supported (float32, float16, bfloat16)")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least one element")
    width = x.shape[-1]
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        if t.shape != (width,):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({width},)")
        if t.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"{name}: dtype {t.dtype}, expected {x.dtype} or float32")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias need the same dtype")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    weight = weight if weight is None else weight.contiguous()
    bias = bias if bias is None else bias.contiguous()
    del device
    if _wants_grad(x, weight, bias):
        return _LayerNorm.apply(x, weight, bias, float(eps))
    return _norm_forward(x, weight, bias, float(eps), False)[0]


# ---------------------------------------------------------------------------
# distance buckets and the dense bias

_buckets: dict = {}


def _bucket_handle(device: torch.device, num_buckets: int, max_distance: int, bidirectional: bool) -> int:
    """The library's handle for one bucket map on one device, made once and
    kept (a few kilobytes each)."""
    key = (device.index, num_buckets, max_distance, bidirectional)
    h = _buckets.get(key)
    if h is None:
        out = C.c_void_p()
        with torch.cuda.device(device):
            status = _lib().fm_buckets_create(C.byref(out), num_buckets, max_distance, int(bidirectional))
        if status == fb.FM_ERR_INVALID_ARG:
            raise ValueError(f"{num_buckets} buckets up to distance {max_distance}: needs 2 to 4096 buckets (even "
                             "and at least 4 where bidirectional) and a max_distance of at most 2048 that is beyond "
                             "the buckets of single distances")
        if status:
            raise fb.FmError(status, "fm_buckets_create")
        h = _buckets.setdefault(key, out.value)
        if h != out.value:  # another thread was first
            _lib().fm_buckets_destroy(out)
    return h


def bucket_map(num_buckets: int, max_distance: int = 128, bidirectional: bool = True,
               device: torch.device | str = "cuda") -> torch.Tensor:
    """Buckets of the offsets (key place minus query place) -max_distance ..
    max_distance, int32 on the host; farther offsets have the end ones'."""
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("bucket_map needs a CUDA device (the map belongs to one)")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    h = _bucket_handle(device, int(num_buckets), int(max_distance), bool(bidirectional))
    out = torch.empty(2 * int(max_distance) + 1, dtype=torch.int32)
    status = _lib().fm_buckets_map(h, out.data_ptr())
    if status:
        raise fb.FmError(status, "fm_buckets_map")
    return out


def _check_table(table, heads=None):
    if table.dim() != 2:
        raise ValueError(f"table has shape {tuple(table.shape)}, expected (num_buckets, heads)")
    if table.dtype not in _TYPES:
        raise TypeError(f"table: dtype {table.dtype} not supported (float32, float16, bfloat16)")
    if heads is not None and table.shape[1] != heads:
        raise ValueError(f"table has {table.shape[1]} heads, q has {heads}")


class _RelativeBias(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, handle, q_len, k_len, q_start):
        ctx.meta = (table.shape, table.dtype, table.device, handle, q_len, k_len, q_start)
        return _relative_bias(table, handle, q_len, k_len, q_start)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        shape, dtype, device, handle, q_len, k_len, q_start = ctx.meta
        dout = dout.contiguous()
        dtable = torch.empty(shape, dtype=dtype, device=device)

        def pack(work, size):
            return _BIAS.pack(shape[1], q_len, k_len, q_start, _TYPES[dtype], handle, 0, 0, dout.data_ptr(),
                              dtable.data_ptr(), work, size)

        size = _lib().fm_relative_bias_workspace(pack(0, 0))
        work = torch.empty(max(size, 0), dtype=torch.uint8, device=device)
        _call("fm_relative_bias_backward", pack(work.data_ptr(), size), device)
        return dtable, None, None, None, None


def _relative_bias(table, handle, q_len, k_len, q_start):
    out = torch.empty(table.shape[1], q_len, k_len, dtype=table.dtype, device=table.device)
    args = _BIAS.pack(table.shape[1], q_len, k_len, q_start, _TYPES[table.dtype], handle, table.data_ptr(),
                      out.data_ptr(), 0, 0, 0, 0)
    _call("fm_relative_bias_forward", args, table.device)
    return out


def relative_bias(table: torch.Tensor, q_len: int, k_len: int, q_start: int | None = None, max_distance: int = 128,
                  bidirectional: bool = True) -> torch.Tensor:
    """The dense position bias (heads, q_len, k_len) of a learned table
    (num_buckets, heads): out[h, i, j] = table[bucket(j - (q_start + i)), h].

    q_start: the first query's place among the keys; None means the queries
    are the last q_len of k_len places. Distances up to half of a side's
    buckets have a bucket each, farther ones share buckets that widen
    logarithmically up to max_distance (at most 2048). Differentiable in the
    table. Add it to scores of your own; attention() reads the table itself.
    """
    _need_cuda(table=table)
    _check_table(table)
    q_len, k_len = int(q_len), int(k_len)
    if q_len < 0 or k_len < 0:
        raise ValueError("q_len and k_len must not be negative")
    q_start = k_len - q_len if q_start is None else int(q_start)
    handle = _bucket_handle(table.device, table.shape[0], int(max_distance), bool(bidirectional))
    table = table.contiguous()
    if _wants_grad(table):
        return _RelativeBias.apply(table, handle, q_len, k_len, q_start)
    return _relative_bias(table, handle, q_len, k_len, q_start)


# ---------------------------------------------------------------------------
# attention

def poll_error(device: torch.device | str = "cuda") -> int:
    """Wait for the device, then take and clear the operators' error status:
    FM_OK, or FM_ERR_KERNEL_TIMEOUT where a bounded wait in a kernel gave up."""
    with torch.cuda.device(torch.device(device)):
        torch.cuda.synchronize()
        return int(_lib().fm_ops_poll_error())


class _Call:
    """What one attention call's passes share besides the tensors."""

    __slots__ = ("scale", "softcap", "causal", "handle", "slopes", "q_docs", "k_docs", "k_lens", "q_start", "prefix",
                 "start_all")


def _strides(t):
    return t.stride(0), t.stride(1), t.stride(2)


def _heads_adjacent(t):
    return t if t.stride(3) == 1 or t.shape[3] == 1 else t.contiguous()


_ZERO3 = (0, 0, 0)


def _attn_pack(c, q, k, v, out, lse, table, dout, dq, dk, dv, dtable, work, size):
    B, Tq, H, D = q.shape
    return _ATTN.pack(
        B, Tq, k.shape[1], H, k.shape[2], D, _TYPES[q.dtype], c.causal, c.scale, c.softcap,
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        *_strides(q), *_strides(k), *_strides(v), *_strides(out), _ptr(lse),
        _ptr(c.q_docs), _ptr(c.k_docs), _ptr(c.k_lens), _ptr(c.q_start), _ptr(c.prefix), c.start_all,
        c.handle, _ptr(table), 0 if table is None else _TYPES[table.dtype], _ptr(c.slopes),
        _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
        *(_ZERO3 if dout is None else _strides(dout)), *(_ZERO3 if dq is None else _strides(dq)),
        *(_ZERO3 if dk is None else _strides(dk)), *(_ZERO3 if dv is None else _strides(dv)),
        _ptr(dtable), work, size)


def _workspace(c, args, backward, device):
    size = _lib().fm_attention_workspace(args, backward)
    return size, (torch.empty(size, dtype=torch.uint8, device=device) if size > 0 else None)


def _attn_forward(c, q, k, v, table, want_lse):
    B, Tq, H, D = q.shape
    out = torch.empty(B, Tq, H, D, dtype=q.dtype, device=q.device)
    lse = torch.empty(B, H, Tq, dtype=torch.float32, device=q.device) if want_lse else None
    args = _attn_pack(c, q, k, v, out, lse, table, None, None, None, None, None, 0, 0)
    size, work = _workspace(c, args, 0, q.device)
    if work is not None:
        args = args[:-16] + struct.pack("=Qq", work.data_ptr(), size)
    _call("fm_attention_forward", args, q.device)
    return out, lse


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, table, c):
        out, lse = _attn_forward(c, q, k, v, table, True)
        ctx.save_for_backward(q, k, v, table, out, lse)
        ctx.c = c
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, _):
        q, k, v, table, out, lse = ctx.saved_tensors
        c = ctx.c
        dout = _heads_adjacent(dout)
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        dtable = None
        if table is not None and ctx.needs_input_grad[3]:
            dtable = torch.empty(table.shape, dtype=table.dtype, device=table.device)
        args = _attn_pack(c, q, k, v, out, lse, table, dout, dq, dk, dv, dtable, 0, 0)
        size, work = _workspace(c, args, 1, q.device)
        if work is not None:
            args = args[:-16] + struct.pack("=Qq", work.data_ptr(), size)
        _call("fm_attention_backward", args, q.device)
        return dq, dk, dv, dtable, None


def _int32(name, t, shape):
    if t is None:
        return None
    if t.dtype != torch.int32:
        raise TypeError(f"{name}: dtype {t.dtype}, expected int32")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    return t.contiguous()


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale: float | None = None, causal: bool = False,
              prefix: torch.Tensor | None = None, softcap: float = 0.0, table: torch.Tensor | None = None,
              max_distance: int = 128, bidirectional: bool = True, slopes: torch.Tensor | None = None,
              q_docs: torch.Tensor | None = None, k_docs: torch.Tensor | None = None,
              k_lens: torch.Tensor | None = None, q_start: int | torch.Tensor | None = None,
              return_lse: bool = False):
    """softmax(z) v over frames, z = scale q.k, capped, biased by distance and
    masked; (batch, q_len, heads, dim) in q's type.

    q: (batch, q_len, heads, dim); k, v: (batch, k_len, kv_heads, dim) with
    heads a multiple of kv_heads (consecutive query heads share a key head).
    float32, float16 or bfloat16, any strides (copied first only where the dim
    elements are not adjacent); dim up to 256.

    scale: 1/sqrt(dim) where None. softcap: z becomes softcap *
    tanh(z / softcap) where above 0. table: learned bias by distance bucket
    (num_buckets, heads), of q's type or float32, with relative_bias()'s
    max_distance and bidirectional. slopes: (heads,) float32, z loses
    slopes[h] * |distance|.

    Query i stands at place q_start + i of the keys' axis (an int, or int32
    (batch,); None: the queries are the last q_len of each row's keys). A key
    is seen where it is below k_lens (int32 (batch,)), carries the query's
    document id (q_docs, k_docs: int32 (batch, len); negative ids are padding)
    and, if causal, is not after the query or lies below prefix (int32
    (batch,)). A query that sees nothing returns zeros and passes no gradient.
    Keys past k_lens and padding frames are never read into a result.

    Differentiable in q, k, v and table (once). return_lse: also the log of
    the softmax's sum, (batch, heads, q_len) float32 (no gradient).
    """
    _need_cuda(q=q, k=k, v=v, table=table, slopes=slopes, q_docs=q_docs, k_docs=k_docs, k_lens=k_lens, prefix=prefix)
    if q.dtype not in _TYPES:
        raise TypeError(f"q: dtype {q.dtype} not supported (float32, float16, bfloat16)")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError(f"q, k and v need one dtype, got {q.dtype}, {k.dtype}, {v.dtype}")
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError(f"q, k, v have shapes {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}; expected "
                         "(batch, q_len, heads, dim) and twice (batch, k_len, kv_heads, dim)")
    B, Tq, H, D = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != D or D < 1 or Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"q {tuple(q.shape)} does not fit k and v {tuple(k.shape)}: same batch and dim, heads a "
                         "multiple of the keys' heads")
    if D > 256:
        raise ValueError(f"dim {D} is not supported (at most 256)")
    c = _Call()
    c.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    c.softcap = float(softcap)
    if not (math.isfinite(c.scale) and c.softcap >= 0 and math.isfinite(c.softcap)):
        raise ValueError("scale must be finite, softcap finite and not negative")
    c.causal = 1 if causal else 0
    if prefix is not None and not causal:
        raise ValueError("prefix needs causal=True")
    if (q_docs is None) != (k_docs is None):
        raise ValueError("q_docs and k_docs go together")
    c.q_docs, c.k_docs = _int32("q_docs", q_docs, (B, Tq)), _int32("k_docs", k_docs, (B, Tk))
    c.k_lens, c.prefix = _int32("k_lens", k_lens, (B,)), _int32("prefix", prefix, (B,))
    c.q_start, c.start_all = None, Q_START_END
    if isinstance(q_start, torch.Tensor):
        _need_cuda(q=q, q_start=q_start)
        c.q_start = _int32("q_start", q_start, (B,))
    elif q_start is not None:
        c.start_all = max(-(1 << 40), min(int(q_start), 1 << 40))
    c.slopes = None
    if slopes is not None:
        if slopes.dtype != torch.float32 or tuple(slopes.shape) != (H,):
            raise ValueError(f"slopes must be float32 of shape ({H},)")
        if slopes.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("slopes are constants: no gradient is computed for them")
        c.slopes = slopes.contiguous()
    c.handle = 0
    if table is not None:
        _check_table(table, H)
        if table.dtype not in (q.dtype, torch.float32):
            raise TypeError(f"table: dtype {table.dtype}, expected {q.dtype} or float32")
        c.handle = _bucket_handle(q.device, table.shape[0], int(max_distance), bool(bidirectional))
        table = table.contiguous()
    q, k, v = _heads_adjacent(q), _heads_adjacent(k), _heads_adjacent(v)
    if _wants_grad(q, k, v, table):
        out, lse = _Attention.apply(q, k, v, table, c)
    else:
        out, lse = _attn_forward(c, q, k, v, table, return_lse)
    return (out, lse) if return_lse else out
