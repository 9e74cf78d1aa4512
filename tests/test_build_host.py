"""When the extension of the attention layers' operators is compiled again (no GPU)."""
import os

import torch

from gated_deltanet_linear_recurrence_gb300 import build as B


def test_another_torch_wants_another_extension(monkeypatch):
    B.build()
    made = os.path.getmtime(B.binding_path())
    B.build()
    assert os.path.getmtime(B.binding_path()) == made  # nothing changed: kept
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert B._binding_stale(B._headers())


def test_a_missing_extension_is_stale(monkeypatch, tmp_path):
    B.build()
    assert not B._binding_stale(B._headers())
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path))
    assert B._binding_stale(B._headers())
