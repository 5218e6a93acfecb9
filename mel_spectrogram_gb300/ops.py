"""Operators of a model over mel frames (include/fm_ops.h): layer norm, a
learned position bias by distance buckets, and attention over frames; and those of
a recurrent block: root-mean-square norm with the residual's addition, a gated
recurrence, and the gated linear layer of its feed-forward part, the first and the
last of them in 8 bits too.

Functions on CUDA tensors with autograd support. Every computation runs in the
library's own kernels, on the current stream of the tensors' device;
``_fm_torch`` (csrc/torch/fm_torch.cpp) checks arguments, allocates outputs and
workspaces and builds the autograd nodes. Bad arguments raise ValueError or
TypeError, a failing library call FmError; second derivatives raise RuntimeError,
forward-mode derivatives and traces NotImplementedError. Inputs, masks included,
that are changed in place before the backward pass raise there.

    y = layer_norm(x, weight, bias)                      # (..., width)
    b = relative_bias(table, q_len, k_len)               # (heads, q_len, k_len)
    o = attention(q, k, v, table=table, q_docs=d, k_docs=d)   # (batch, len, heads, dim)
    y, x = rms_norm(x, weight, residual)                 # (..., width), twice
    h, state = gated_scan(x, gate, state, return_state=True)  # (batch, frames, channels)
    h = gated_linear(x, w_gate, w_up)                    # (..., hidden)
"""
from __future__ import annotations

import ctypes as C
import os

import torch

from . import _binding as fb

if not os.path.exists(fb.LIB_PATH):
    fb.lib()  # raises with the build command

try:
    from . import _fm_torch as _C  # noqa: E402
except ImportError as e:
    raise ImportError(f"the operators' binding to torch does not load ({e}): build it with "
                      "`python -m mel_spectrogram_gb300.build` where torch is installed") from e

_C.set_error(fb.FmError)

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
    "fm_rms_norm_forward",
    "fm_rms_norm_backward",
    "fm_rms_norm_workspace",
    "fm_rows_8bit",
    "fm_gated_forward",
    "fm_gated_backward",
    "fm_gated_workspace",
    "fm_scan_forward",
    "fm_scan_backward",
    "fm_scan_marks",
    "fm_scan_workspace",
    "fm_ops_poll_error",
    "fm_ops_selftest_wait",
]


def library() -> C.CDLL:
    """The library with the prototypes of fm_ops.h, for calls by pointer (always
    the release build: the debug build holds the mel kernels only)."""
    L = fb.load(fb.LIB_PATH)
    vp, ci = C.c_void_p, C.c_int
    for op in ("layer_norm", "relative_bias", "attention"):
        for way in ("forward", "backward"):
            f = getattr(L, f"fm_{op}_{way}")
            f.argtypes, f.restype = [vp, vp], ci
        f = getattr(L, f"fm_{op}_workspace")
        f.argtypes, f.restype = [vp] + ([ci] if op == "attention" else []), C.c_int64
    for name in ("fm_rms_norm_forward", "fm_rms_norm_backward", "fm_rows_8bit", "fm_gated_forward",
                 "fm_gated_backward", "fm_scan_forward", "fm_scan_backward"):
        f = getattr(L, name)
        f.argtypes, f.restype = [vp, vp], ci
    for name in ("fm_rms_norm_workspace", "fm_scan_marks", "fm_scan_workspace"):
        f = getattr(L, name)
        f.argtypes, f.restype = [vp], C.c_int64
    L.fm_gated_workspace.argtypes, L.fm_gated_workspace.restype = [vp, ci], C.c_int64
    L.fm_buckets_create.argtypes, L.fm_buckets_create.restype = [C.POINTER(vp), ci, ci, ci], ci
    L.fm_buckets_map.argtypes, L.fm_buckets_map.restype = [vp, vp], ci
    L.fm_buckets_destroy.argtypes, L.fm_buckets_destroy.restype = [vp], ci
    L.fm_ops_poll_error.argtypes, L.fm_ops_poll_error.restype = [], ci
    L.fm_ops_selftest_wait.argtypes, L.fm_ops_selftest_wait.restype = [vp], ci
    return L


def _cuda_device(device) -> torch.device:
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("the operators run only on the GPU: a CUDA device is needed")
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of x over its last dimension, in x's type.

    x: (..., width) float32, float16 or bfloat16, any strides (rows whose
    elements are not adjacent are copied first). weight, bias: (width,), of
    x's type or float32 (both the same type), or None for ones and zeros.
    Statistics are 32-bit: the mean, then the mean squared deviation from it.
    Differentiable in x, weight and bias (once).
    """
    return _C.layer_norm(x, weight, bias, eps)


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
             eps: float = 1e-6):
    """Root-mean-square norm over the last dimension, total / sqrt(mean(total^2) +
    eps) * weight in x's type; with a residual, (that, total).

    total is x + residual, rounded to their type (x itself without one): the
    stream that the next addition takes. x, residual: (..., width) float32,
    float16 or bfloat16, both the same, any strides (rows whose elements are not
    adjacent are copied first). weight: (width,), of x's type or float32, or None
    for ones. The mean of squares is 32-bit (magnitudes beyond 1e18
    overflow it, those below 1e-18 vanish in it: with an eps of 0 their norm is infinite).
    Differentiable in x, weight and residual (once); total's own gradient is added
    in the same pass.
    """
    return _C.rms_norm(x, weight, residual, eps)


def rms_norm_8bit(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                  eps: float = 1e-6):
    """rms_norm in 8 bits: (values, scales), with a residual (values, scales, total).

    values: (..., width) float8_e4m3fn, scales: (...) float32, one a row: the row's
    largest magnitude / 448 (at least 2^-126); values * scale is the norm, rounded
    once from 32 bits. A row that holds an infinity or NaN gets a scale of NaN. For
    serving: it has no gradient, and raises RuntimeError where one is wanted.
    """
    return _C.rms_norm_8bit(x, weight, residual, eps)


def rows_8bit(x: torch.Tensor):
    """x (..., width) in 8 bits, rows by rows: (values, scales) as rms_norm_8bit's."""
    return _C.rows_8bit(x)


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu") -> torch.Tensor:
    """act(x w_gate^T) * (x w_up^T), the first half of a gated feed-forward part, in
    one kernel; in x's type.

    x: (..., width), w_gate, w_up: (hidden, width), as torch.nn.Linear holds them;
    float32, float16 or bfloat16, all the same, any strides (rows whose elements are
    not adjacent are copied first). activation: "silu", "gelu" (by erf), "sigmoid" or
    "relu". Sums are 32-bit, and the product is rounded once.

    Differentiable in x, w_gate and w_up (once). Nothing but them is kept for the
    backward pass, which works the two projections out again; their gradients are
    rounded to the tensors' type before the products with the weights and with x.
    """
    return _C.gated_linear(x, w_gate, w_up, activation)


def gated_linear_8bit(x: torch.Tensor, x_scales: torch.Tensor, w_gate: torch.Tensor, gate_scales: torch.Tensor,
                      w_up: torch.Tensor, up_scales: torch.Tensor, activation: str = "silu",
                      dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """gated_linear of 8-bit rows, in dtype (bfloat16, float16 or float32).

    x: (..., width) float8_e4m3fn with x_scales (...) float32, as rms_norm_8bit gives
    them; w_gate, w_up: (hidden, width) float8_e4m3fn with gate_scales, up_scales
    (hidden,), as rows_8bit gives them. For serving: it has no gradient, and raises
    RuntimeError where one is wanted.
    """
    return _C.gated_linear_8bit(x, x_scales, w_gate, gate_scales, w_up, up_scales, activation, dtype)


def gated_scan(x: torch.Tensor, gate: torch.Tensor, state: torch.Tensor | None = None, *,
               lens: torch.Tensor | None = None, docs: torch.Tensor | None = None, reverse: bool = False,
               return_state: bool = False):
    """Gated linear recurrence over frames, h_t = a_t h_(t-1) + (1 - a_t) x_t with
    a_t = sigmoid(gate_t), each channel by itself; h in x's type.

    x, gate: (batch, frames, channels) float32, float16 or bfloat16, both the same,
    any strides (copied first only where channels are not adjacent). state: float32
    (batch, channels), where the recurrence starts; None for zeros. It is held in 32
    bits throughout. reverse: the frames are walked from the last to the first.

    lens: int32 (batch,), frames in use of each row. docs: int32 (batch, frames)
    document ids; negative ids are padding. Frames that are not in use return 0,
    pass no gradient, leave the state as it is, and may hold anything. The first frame
    of the walk goes on from `state`; where a later one's id differs from the id
    before it, the recurrence starts from 0.

    return_state: (h, the state after the walk, float32). Differentiable in x, gate
    and state (once).
    """
    return _C.gated_scan(x, gate, state, lens, docs, reverse, return_state)


def bucket_map(num_buckets: int, max_distance: int = 128, bidirectional: bool = True,
               device: torch.device | str = "cuda") -> torch.Tensor:
    """Buckets of the offsets (key place minus query place) -max_distance ..
    max_distance, int32 on the host; farther offsets have the end ones'."""
    device = _cuda_device(device)
    handle = _C.buckets(device.index, num_buckets, max_distance, bidirectional)
    out = torch.empty(2 * int(max_distance) + 1, dtype=torch.int32)
    status = library().fm_buckets_map(handle, out.data_ptr())
    if status:
        raise fb.FmError(status, "fm_buckets_map")
    return out


def relative_bias(table: torch.Tensor, q_len: int, k_len: int, q_start: int | None = None, max_distance: int = 128,
                  bidirectional: bool = True) -> torch.Tensor:
    """The dense position bias (heads, q_len, k_len) of a learned table
    (num_buckets, heads): out[h, i, j] = table[bucket(j - (q_start + i)), h].

    q_start: the first query's place among the keys; None means the queries
    are the last q_len of k_len places. Distances up to half of a side's
    buckets have a bucket each, farther ones share buckets that widen
    logarithmically up to max_distance (at most 2048). Differentiable in the
    table (once). Add it to scores of your own; attention() reads the table
    itself.
    """
    return _C.relative_bias(table, q_len, k_len, q_start, max_distance, bidirectional)


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

    Where a wait inside a kernel gave up (after two seconds; never in ordinary
    running) that call's results are not valid, and the next calls raise FmError
    until poll_error() has taken the error.

    Differentiable in q, k, v and table (once). return_lse: also the log of
    the softmax's sum, (batch, heads, q_len) float32 (no gradient).
    """
    return _C.attention(q, k, v, scale, causal, prefix, softcap, table, max_distance, bidirectional, slopes, q_docs,
                        k_docs, k_lens, q_start, return_lse)


def poll_error(device: torch.device | str = "cuda") -> int:
    """Wait for the device, then take and clear the operators' error status:
    FM_OK, or FM_ERR_KERNEL_TIMEOUT where a bounded wait in a kernel of attention(),
    gated_linear() or gated_scan() gave up. Until it is taken those that would wait,
    and their backward passes, raise it; after replays of a recorded graph, which
    make no call, ask here."""
    with torch.cuda.device(_cuda_device(device)):
        return int(library().fm_ops_poll_error())
