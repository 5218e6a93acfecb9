"""The gated recurrence's workspace through the C ABI: what is too small for its sums, or
not asked for at all, is left as it is."""
from __future__ import annotations

import ctypes as C

import pytest
import torch

from tests import recurrent_reference as ref
from tests import test_recurrent_abi_gpu as abi
from tests import test_recurrent_gpu as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from mel_spectrogram_gb300 import ops

    return ops.library()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 2416, 16), (2, 4095, 8), (1, 1000, 80), (1, 600, 8200), (9, 4096, 1024)])
def test_no_workspace_is_needed(L, shape, dtype):
    B, T, Cn = shape
    x, gate, state = (t.contiguous() for t in base.inputs(shape, dtype, 7))
    g = base.gen(2)
    dy, dend = base.randn(g, *shape, dtype=dtype), base.randn(g, B, Cn)
    s, got = (T * Cn, Cn), []
    for room in (0, 16, 4096):
        y, dx, dg = (torch.empty_like(x) for _ in range(3))
        end, dstate = torch.empty_like(state), torch.empty_like(state)
        common = dict(batch=B, frames=T, channels=Cn, dtype=abi.CODES[dtype], x=x, gate=gate, x_s=s, gate_s=s)
        a = abi.fill("fm_scan_args", **common, state=state, end=end, y=y, y_s=s)
        b = abi.fill("fm_scan_args", **common, dy=dy, dy_s=s, dend=dend, dx=dx, dx_s=s, dgate=dg, dgate_s=s, dstate=dstate)
        assert L.fm_scan_workspace(C.byref(a)) == L.fm_scan_workspace(C.byref(b)) == 0
        marks = torch.empty(L.fm_scan_marks(C.byref(a)), dtype=torch.uint8, device="cuda")
        work = torch.full((1 << 20,), 0xff, dtype=torch.uint8, device="cuda")  # far more than it is said to hold
        for args, call in ((a, L.fm_scan_forward), (b, L.fm_scan_backward)):
            args.marks = marks.data_ptr()
            args.workspace, args.workspace_bytes = work.data_ptr(), room
            abi.run(call, args, None)
        assert (work == 0xff).all()
        got.append((y, end, dx, dg, dstate))
    for other in got[1:]:
        assert all(torch.equal(u, v) for u, v in zip(got[0], other))
    if B * T * Cn < 10 ** 5:
        want = ref.scan(x, gate, state, dy=dy, dend=dend)
        for name, t in zip(("out", "state", "dx", "dgate", "dstate"), got[0]):
            ref.close(t, *want[name], name)
