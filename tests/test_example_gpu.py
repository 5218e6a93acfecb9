"""The frame-encoder example: it learns, and streams what it predicts in packs."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "frame_encoder.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("frame_encoder", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# two blocks, each with about ten roundings to the type on the way to the
# prediction, which differ in order between the two forms: within 32 roundings
@pytest.mark.parametrize("dtype,room", [(torch.float32, 1e-4), (torch.bfloat16, 32 * 2.0 ** -9)])
def test_learns_and_streams(example, dtype, room):
    losses, far = example.run(steps=12, dtype=dtype, seconds=1.0)
    assert losses[-1] < 0.5 * losses[0], losses
    assert far < room


def test_packed_rows_are_apart(example):
    # a recording's predictions do not depend on what it is packed with
    torch.manual_seed(1)
    model = example.FrameModel().to("cuda", torch.float32)
    frames = [torch.randn(n, 80, device="cuda") for n in (70, 140, 33)]
    with torch.no_grad():
        batch, ids = example.pack(frames, rows=1)
        together = model(batch, ids)
        alone = model(frames[1][None], torch.zeros(1, 140, dtype=torch.int32, device="cuda"))
    assert torch.allclose(together[:, 70:210], alone, rtol=1e-4, atol=1e-4)
