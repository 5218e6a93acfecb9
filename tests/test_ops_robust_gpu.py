"""The frame-encoder operators where calls are easily answered wrongly: many
broken rows at once, large caps, inputs changed between the passes, second
derivatives, first uses inside a recording, waits that give up."""
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


def passes(ops, q, k, v, dy, **kw):
    """The output and the gradients of q, k, v (and a table)."""
    leaves = [t.detach().requires_grad_() for t in (q, k, v)]
    if kw.get("table") is not None:
        kw["table"] = kw["table"].detach().requires_grad_()
        leaves.append(kw["table"])
    out = ops.attention(*leaves[:3], **kw)
    return [out.detach(), *torch.autograd.grad(out, leaves, dy)]


# ---------------------------------------------------------------------------
# more tiles with results that are not finite than there are SMs: a block of
# the second launch works on several of them in turn

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_broken_tiles(ops, dtype, dim):
    B, T = 80, 200  # 320 blocks forward, 640 and 320 backward
    q, k, v, dy, _ = base.make((B, T, T, 4, 2, dim), dtype)
    ids = base.docs_of(T, *[[(0, 90), (1, 70), (2, 40)]] * B)
    clean = passes(ops, q, k, v, dy, q_docs=ids, k_docs=ids)
    broken = [t.clone() for t in (q, k, v, dy)]
    for t in broken:
        t[:, 90:160, :, 3] = math.inf
    again = []
    for _ in range(2):
        got = passes(ops, *broken, q_docs=ids, k_docs=ids)
        again.append(got)
        for g, want in zip(got, clean):
            # f16's dS has another power of two without the broken recording
            for part in (slice(0, 90), slice(160, T)):
                room = 2 * ref.U[dtype] * want[:, part].abs().max()
                assert ((g[:, part] - want[:, part]).abs() <= room).all()
            assert not torch.isfinite(g[:, 90:160]).all()
        assert torch.equal(got[0][:, :90], clean[0][:, :90]) and torch.equal(got[0][:, 160:], clean[0][:, 160:])
    for a, b in zip(*again):
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
    # causal: every row's last keys are broken
    clean = passes(ops, q, k, v, dy, causal=True)
    v2 = v.clone()
    v2[:, 150:] = math.nan
    got = passes(ops, q, k, v2, dy, causal=True)
    assert torch.equal(got[0][:, :150], clean[0][:, :150]) and got[0][:, 150:].isnan().all()
    room = 2 * ref.U[dtype] * clean[1][:, :150].abs().max()
    assert ((got[1][:, :150] - clean[1][:, :150]).abs() <= room).all()
    assert ops.poll_error() == 0


# ---------------------------------------------------------------------------
# second derivatives are refused, not dropped

def test_second_derivatives(ops):
    q, k, v, _, g = base.make((1, 6, 6, 2, 1, 16), F32)
    x, w = base.randn(g, 5, 16), base.randn(g, 16)
    table = base.randn(g, 8, 2)
    calls = [(lambda x, w: ops.layer_norm(x, w), (x, w)),
             (lambda t: ops.relative_bias(t, 4, 5, max_distance=16), (table,)),
             (lambda q, k, v, t: ops.attention(q, k, v, table=t, max_distance=16), (q, k, v, table))]
    for call, inputs in calls:
        leaves = [t.clone().requires_grad_() for t in inputs]
        first = torch.autograd.grad(call(*leaves).square().sum(), leaves, create_graph=True)
        for d in first:
            assert d.requires_grad
            # beside a term that has a derivative, as in a gradient penalty
            with pytest.raises(RuntimeError, match="differentiable once"):
                torch.autograd.grad(d.square().sum() + leaves[0].square().sum(), leaves, retain_graph=True,
                                    allow_unused=True)
    # the bias's gradient does not depend on the table: a constant where the gradient given is one
    leaf = table.clone().requires_grad_()
    (d,) = torch.autograd.grad(ops.relative_bias(leaf, 4, 5, max_distance=16).sum(), leaf, create_graph=True)
    (second,) = torch.autograd.grad((d * leaf).sum(), leaf)
    assert torch.equal(second, d)


# ---------------------------------------------------------------------------
# caps far above the scores, and scores on both sides of them

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("softcap", [200.0, 1e4, 1e6, 1e8, 1e30])
@pytest.mark.parametrize("Tq", [1, 4, 16, 129])
def test_large_caps(ops, Tq, softcap, dtype):
    q, k, v, dy, _ = base.make((2, Tq, 150, 4, 2, 64), dtype)
    base.check_attention(ops, q, k, v, f"cap {softcap}", softcap=softcap, scale=0.5)
    base.check_attention(ops, q, k, v, f"cap {softcap}", dy=dy, softcap=softcap, scale=0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("softcap", [1e-46, 1e-39, 1e-20, 1e-3])
@pytest.mark.parametrize("Tq", [4, 129])
def test_small_caps(ops, Tq, softcap, dtype):
    q, k, v, dy, _ = base.make((1, Tq, 150, 2, 2, 64), dtype)
    q[:, 1] = 0  # scores of 0 beside others far beyond the cap
    base.check_attention(ops, q, k, v, f"cap {softcap}", softcap=softcap)
    base.check_attention(ops, q, k, v, f"cap {softcap}", dy=dy, softcap=softcap)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("softcap", [30.0, 1e4])
@pytest.mark.parametrize("Tq", [3, 129])
def test_caps_between_rows(ops, Tq, softcap, dtype):
    # one query whose scores reach the cap beside others far below it
    q, k, v, dy, _ = base.make((1, Tq, 150, 2, 2, 64), dtype)
    q[:, 1] *= softcap / 8
    base.check_attention(ops, q, k, v, f"cap {softcap}", softcap=softcap)
    base.check_attention(ops, q, k, v, f"cap {softcap}", dy=dy, softcap=softcap)


# ---------------------------------------------------------------------------
# masks and slopes changed between the passes

def test_changed_masks_are_noticed(ops):
    q, k, v, dy, g = base.make((2, 20, 20, 2, 2, 64), BF16)
    ids = base.docs_of(20, [(0, 20)], [(0, 12), (1, 8)])
    extra = {"q_docs": ids, "k_docs": ids.clone(), "k_lens": base.lengths(20, 15), "q_start": base.lengths(0, 1),
             "prefix": base.lengths(3, 4), "slopes": torch.rand(2, device="cuda", generator=g)}
    for name in extra:
        kw = {n: t.clone() for n, t in extra.items()}
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        out = ops.attention(*leaves, causal=True, **kw)
        want = torch.autograd.grad(out, leaves, dy, retain_graph=True)
        kw[name].add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            torch.autograd.grad(out, leaves, dy)
        del out, want


# ---------------------------------------------------------------------------
# forward-mode derivatives are refused, not dropped

def test_forward_mode(ops):
    import torch.autograd.forward_ad as fw

    q, k, v, _, g = base.make((1, 6, 6, 2, 1, 16), F32)
    x, w, table = base.randn(g, 5, 16), base.randn(g, 16), base.randn(g, 8, 2)
    calls = [(lambda x, w: ops.layer_norm(x, w), (x, w)),
             (lambda x, b: ops.layer_norm(x, None, b), (x, w)),
             (lambda t: ops.relative_bias(t, 4, 5, max_distance=16), (table,)),
             (lambda q, k, v, t: ops.attention(q, k, v, table=t, max_distance=16), (q, k, v, table)),
             (lambda q, k, v, s: ops.attention(q, k, v, slopes=s), (q, k, v, torch.ones(2, device="cuda")))]
    for call, inputs in calls:
        for n in range(len(inputs)):
            for grad in (True, False):
                with fw.dual_level(), torch.set_grad_enabled(grad):
                    args = list(inputs)
                    args[n] = fw.make_dual(args[n], torch.ones_like(args[n]))
                    with pytest.raises(NotImplementedError, match="forward-mode"):
                        call(*args)
                    call(*inputs)  # no tangent: as ever


# ---------------------------------------------------------------------------
# traces, which would hold the allocations alone, are refused

@pytest.mark.filterwarnings("ignore")
def test_traces(ops):
    from torch.fx.experimental.proxy_tensor import make_fx

    q, k, v, _, g = base.make((1, 6, 6, 2, 1, 16), F32)
    table = base.randn(g, 8, 2)
    for call, inputs in [(lambda x: ops.layer_norm(x), (q,)), (lambda t: ops.relative_bias(t, 4, 5, max_distance=16), (table,)),
                         (lambda q, k, v: ops.attention(q, k, v), (q, k, v))]:
        with pytest.raises(NotImplementedError, match="trac"):
            torch.jit.trace(call, inputs)
        with pytest.raises(NotImplementedError, match="trac"):
            make_fx(call)(*inputs)


# ---------------------------------------------------------------------------
# bucket maps first used where nothing has made them yet

def test_first_use_inside_a_recording(ops):
    q, k, v, dy, g = base.make((1, 40, 40, 2, 2, 64), BF16)
    table = base.randn(g, 38, 2, dtype=BF16)
    ops.attention(q, k, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.attention(q, k, v, table=table, max_distance=77)
        bias = ops.relative_bias(table, 5, 6, max_distance=78)
    graph.replay()
    ref.close(out, *ref.attention(q, k, v, table=table, max_distance=77)["out"], "replayed")
    ref.close(bias, *ref.dense_bias(table, 5, 6, 1, 78, True)["out"], "replayed")


def test_first_use_on_another_stream(ops):
    g = base.gen(3)
    table = base.randn(g, 40, 2)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    torch.cuda._sleep(10 ** 8)  # the default stream is busy: nothing of the other may wait for or pass it
    with torch.cuda.stream(side):
        for far in range(100, 160):
            got.append(ops.relative_bias(table, 30, 200, max_distance=far))
    side.synchronize()
    for far, out in zip(range(100, 160), got):
        ref.close(out, *ref.dense_bias(table, 30, 200, 170, far, True)["out"], f"max_distance {far}")


# ---------------------------------------------------------------------------
# what a mask hides changes no bit of the others, however large it is

def interleaved(dtype, dim):
    """Two recordings frame by frame in turn, so that every tile and warp holds
    both: inputs, the same with the second one loud, and the ids."""
    T = 300
    ids = (torch.arange(T, dtype=torch.int32, device="cuda") % 2)[None]
    q, k, v, dy, _ = base.make((1, T, T, 2, 1, dim), dtype)
    k = k * torch.linspace(0.5, 4, T, device="cuda").to(dtype)[None, :, None, None]  # maxima that rise from tile to tile
    loud = [t.clone() for t in (q, k, v, dy)]
    for t, f in zip(loud, (4, 8, 30, 300)):
        t[:, 1::2] *= f
    return (q, k, v, dy), loud, ids


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_hidden_rows_change_no_output(ops, dtype, dim, softcap):
    plain, loud, ids = interleaved(dtype, dim)
    for causal in (False, True):
        for rows in (slice(0, 300), slice(150, 153)):  # in tiles, and few
            want, got = (ops.attention(q[:, rows], k, v, q_docs=ids[:, rows], k_docs=ids, causal=causal,
                                       q_start=rows.start, softcap=softcap) for q, k, v, _ in (plain, loud))
            assert torch.equal(got[:, ::2], want[:, ::2])
            assert not torch.equal(got[:, 1::2], want[:, 1::2])


# ---------------------------------------------------------------------------
# nor of their gradients

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_hidden_rows_change_no_gradient(ops, dtype, dim, softcap):
    plain, loud, ids = interleaved(dtype, dim)
    for causal in (False, True):
        want, got = (passes(ops, *inputs, q_docs=ids, k_docs=ids, causal=causal, softcap=softcap)
                     for inputs in (plain, loud))
        for name, a, b in zip(("out", "dq", "dk", "dv"), got, want):
            assert torch.equal(a[:, ::2], b[:, ::2]), (name, causal)
            assert not torch.equal(a[:, 1::2], b[:, 1::2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_later_rows_change_no_gradient(ops, dtype, dim):
    T, n = 300, 150
    q, k, v, dy, _ = base.make((1, T, T, 2, 1, dim), dtype)
    want = passes(ops, q, k, v, dy, causal=True)
    loud = [t.clone() for t in (q, k, v, dy)]
    for t, f in zip(loud, (4, 4, 30, 300)):
        t[:, n:] *= f
    got = passes(ops, *loud, causal=True)
    for a, b in zip(got[:2], want[:2]):  # earlier queries' output and gradient
        assert torch.equal(a[:, :n], b[:, :n])
    loud = [q.clone(), k, v, dy.clone()]
    loud[0][:, :n] *= 4
    loud[3][:, :n] *= 300
    got = passes(ops, *loud, causal=True)
    for a, b in zip(got[2:], want[2:]):  # later keys' gradients
        assert torch.equal(a[:, n:], b[:, n:])


def test_loud_and_quiet_gradients(ops):
    # f16 rows whose gradients are 10^5 times apart, each within its own bound
    q, k, v, dy, _ = base.make((1, 200, 200, 2, 1, 64), F16)
    ids = base.docs_of(200, [(0, 100), (1, 100)])
    dy[:, :100] *= 2 ** -5
    v[:, :100] *= 2 ** -2
    dy[:, 100:] *= 300
    v[:, 100:] *= 30
    base.check_attention(ops, q, k, v, "loud and quiet", dy=dy, q_docs=ids, k_docs=ids)


# ---------------------------------------------------------------------------
# the error word

def test_poll_waits_for_every_stream(ops):
    side, event = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(5 * 10 ** 8)
        event.record()
    assert ops.library().fm_ops_poll_error() == 0
    assert event.query()


def test_a_wait_that_gave_up_is_raised(ops):
    from mel_spectrogram_gb300 import FM_ERR_KERNEL_TIMEOUT, FM_OK, FmError

    for dtype in TYPES:
        q, k, v, dy, _ = base.make((1, 140, 140, 2, 2, 64), dtype)
        want = passes(ops, q, k, v, dy)
        leaf = q.detach().requires_grad_()
        out = ops.attention(leaf, k, v)
        side = torch.cuda.Stream()
        assert ops.library().fm_ops_selftest_wait(side.cuda_stream) == FM_OK
        side.synchronize()
        for _ in range(2):
            with pytest.raises(FmError) as e:
                ops.attention(q, k, v)
            assert e.value.status == FM_ERR_KERNEL_TIMEOUT
        with pytest.raises(RuntimeError, match="KERNEL_TIMEOUT"):
            torch.autograd.grad(out, leaf, dy)
        assert ops.poll_error() == FM_ERR_KERNEL_TIMEOUT
        assert ops.poll_error() == FM_OK
        assert all(torch.equal(a, b) for a, b in zip(want, passes(ops, q, k, v, dy)))


# ---------------------------------------------------------------------------
# arguments whose truth value is an error

def test_flags_without_a_truth_value(ops):
    q = torch.randn(1, 3, 2, 8, device="cuda")
    t = torch.randn(8, 2, device="cuda")
    many = torch.ones(2)
    for call in (lambda: ops.attention(q, q, q, causal=many), lambda: ops.attention(q, q, q, bidirectional=many),
                 lambda: ops.attention(q, q, q, return_lse=many),
                 lambda: ops.relative_bias(t, 3, 3, max_distance=9, bidirectional=many),
                 lambda: ops.bucket_map(8, 9, many)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()


# ---------------------------------------------------------------------------
# partial bias gradients beyond 2^32 of a bucket's elements

def test_bias_gradient_of_many_rows(ops):
    # 65535 batch entries x 33 tiles of queries x 2048 offsets of one bucket; 35 GB of partial sums
    B, Tq = 65535, 2100
    q = torch.zeros(B, Tq, 1, 1, device="cuda")
    k = torch.zeros(1, 2, 1, 1, device="cuda").expand(B, 2, 1, 1)
    v = torch.tensor([1.0, 0.0], device="cuda").view(1, 2, 1, 1).expand(B, 2, 1, 1)
    dy = torch.zeros(B, Tq, 1, 1, device="cuda")
    dy[-1000:] = 1.0
    table = torch.zeros(4, 1, device="cuda", requires_grad=True)
    out = ops.attention(q, k, v, table=table, max_distance=2048, q_start=0)
    (d,) = torch.autograd.grad(out, table, dy)
    # weights of 1/2: dS is 1/4 and -1/4; bucket 1 gets all pairs but (0, 0), (1, 1) and (0, 1), bucket 3 the last
    assert d.flatten().tolist() == [0.0, 250.0, 0.0, -250.0]
    del q, k, v, dy, out
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# tensors without memory of their own: an absent pointer must not read as an
# absent argument

class Wrapper(torch.Tensor):
    """A subclass around another tensor, as distributed and fake tensors are."""

    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_wrapper_subclass(cls, t.shape, dtype=t.dtype, device=t.device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


def test_tensors_without_memory(ops):
    from torch._subclasses.fake_tensor import FakeTensorMode

    x, w = torch.randn(5, 16, device="cuda"), torch.randn(16, device="cuda")
    q, k, v, _, g = base.make((2, 6, 6, 2, 1, 16), F32)
    ids = torch.zeros(2, 6, dtype=torch.int32, device="cuda")
    table = base.randn(g, 8, 2)
    extra = {"q_docs": ids, "k_docs": ids, "k_lens": base.lengths(3, 4), "q_start": base.lengths(0, 1),
             "prefix": base.lengths(3, 4), "slopes": torch.rand(2, device="cuda"), "table": table}
    calls = [lambda: ops.layer_norm(x, Wrapper(w)), lambda: ops.layer_norm(x, w, Wrapper(w)),
             lambda: ops.layer_norm(Wrapper(x), w), lambda: ops.relative_bias(Wrapper(table), 4, 5, max_distance=16),
             lambda: ops.attention(Wrapper(q), k, v)]
    for name in extra:
        kw = dict(extra, **{name: Wrapper(extra[name])})
        calls.append(lambda kw=kw: ops.attention(q, k, v, causal=True, max_distance=16, **kw))
    for call in calls:
        with pytest.raises(ValueError, match="memory"):
            call()
    with FakeTensorMode(allow_non_fake_inputs=True):
        for call in (lambda: ops.layer_norm(x, w), lambda: ops.relative_bias(table, 4, 5, max_distance=16),
                     lambda: ops.attention(q, k, v)):
            with pytest.raises(ValueError, match="memory"):
                call()


# ---------------------------------------------------------------------------
# views whose sign is a flag

def test_negated_views(ops):
    def same(call, inputs, dy):
        for n in range(len(inputs) + 1):
            got = []
            for flip in (lambda t: torch._neg_view(t), lambda t: -t):
                args = [flip(t) if m == n else t.clone() for m, t in enumerate(inputs)]
                leaves = [t.detach().requires_grad_() for t in args]
                out = call(*leaves)
                got.append([out.detach(), *torch.autograd.grad(out, leaves, flip(dy) if n == len(inputs) else dy),
                            call(*args)])
            for a, b in zip(*got):
                assert torch.equal(a, b), n

    q, k, v, dy, g = base.make((1, 40, 40, 2, 2, 64), BF16)
    table = base.randn(g, 8, 2, dtype=BF16)
    same(lambda x, w, b: ops.layer_norm(x, w, b), [base.randn(g, 7, 64), base.randn(g, 64), base.randn(g, 64)],
         base.randn(g, 7, 64))
    same(lambda t: ops.relative_bias(t, 4, 5, max_distance=16), [table], base.randn(g, 2, 4, 5, dtype=BF16))
    same(lambda q, k, v, t: ops.attention(q, k, v, table=t, max_distance=16), [q, k, v, table], dy)
    slopes = torch.rand(2, device="cuda")
    assert torch.equal(ops.attention(q, k, v, slopes=torch._neg_view(slopes)), ops.attention(q, k, v, slopes=-slopes))
