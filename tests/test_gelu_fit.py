"""The polynomial behind gelu's integral of the tensor-core kernels, from the kernels' source, in
64 bits: as far from the normal distribution's integral as the comment beside it says."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest

from mel_spectrogram_gb300 import build

special = pytest.importorskip("scipy.special")


def test_error_is_what_is_said():
    with open(os.path.join(build.CSRC, "fm_ops_gated_tc.cuh")) as f:
        source = f.read()
    at = source.index("normal_integrals(float2 g")
    said = float(re.findall(r"least relative error up to \|g\| = 14 \(([\d.e-]+)", source[:at])[-1])
    body = source[at:source.index("\n}", at)]
    coefficients = [float(np.float32(c)) for c in re.findall(r"-?\d\.\d+(?=f[,}])", body[:body.index("};") + 1])]
    slope = float(np.float32(re.search(r"both\((0\.304\d+)f\)", body).group(1)))
    assert len(coefficients) == 8
    g = np.linspace(0, 14, 400001)
    t = 1 / (1 + slope * g)
    # both sides without their common factor exp(-g^2 / 2)
    off = np.polyval(coefficients[::-1], t) * t / (0.5 * special.erfcx(g / np.sqrt(2))) - 1
    assert 0.9 * said < np.abs(off).max() <= said
