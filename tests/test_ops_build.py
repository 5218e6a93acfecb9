"""The binding of the frame-encoder operators follows the torch it is built
against."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from mel_spectrogram_gb300 import build as b

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_another_torch_makes_the_binding_stale(monkeypatch, tmp_path):
    b.build()
    identity = b._torch_identity()
    out = os.path.join(b.BUILD, "fm_torch.cpp.o")
    assert not b._torch_stale(out, identity)
    assert b._torch_stale(out, identity.replace("__version__ = '", "__version__ = '9"))
    assert b._torch_stale(str(tmp_path / "none.o"), identity)
    monkeypatch.setattr(b, "_torch_identity", lambda: "")
    assert b._compile_torch() == ""  # no torch: no binding
    # an object of before there was a note beside it
    (tmp_path / "old.o").write_text("")
    assert b._torch_stale(str(tmp_path / "old.o"), identity)


def test_missing_binding_names_the_build():
    code = """
import sys
class Hide:
    def find_spec(self, name, path=None, target=None):
        if name == "mel_spectrogram_gb300._fm_torch":
            raise ModuleNotFoundError(name)
sys.meta_path.insert(0, Hide())
import mel_spectrogram_gb300
try:
    mel_spectrogram_gb300.attention
except ImportError as e:
    assert "python -m mel_spectrogram_gb300.build" in str(e), e
    print("named")
"""
    b.build()
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.stdout == "named\n", r.stdout + r.stderr
