"""Rows in 8 bits to the bit: the row's largest magnitude / 448, and each value divided by it,
rounded once to 32 bits and once to 8."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from mel_spectrogram_gb300 import ops

    return ops


# by 16 bytes, element by element, and rows wider than registers; enough values that some lie
# next to the middle between two steps
@pytest.mark.parametrize("rows,width", [(32768, 1024), (16384, 1023), (2048, 8200)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_quotients(ops, rows, width, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, width, device="cuda", generator=g).to(dtype)
    size = torch.arange(rows, device="cuda") % 21 - 10
    if dtype is not torch.float16:
        size[7::13], size[8::13], size[9::13] = 100, -80, -120
    x *= torch.exp2(size.float())[:, None].to(dtype)
    values, scales = ops.rows_8bit(x)
    # the host's division: correctly rounded whatever the device's would be
    want = torch.from_numpy(x.float().abs().amax(-1).cpu().numpy() / torch.tensor(448.0).numpy())
    assert torch.equal(scales.cpu(), want.clamp(min=2.0 ** -126))
    want = torch.from_numpy(x.float().cpu().numpy() / scales.cpu().numpy()[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(values.cpu().view(torch.uint8), want.view(torch.uint8))
