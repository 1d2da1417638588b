"""What __graft_entry__.build() needs for what: the C library and the oracle are
built first, and without torch they are all that is built."""
import sys

import pytest


@pytest.fixture
def steps(monkeypatch):
    import __graft_entry__ as entry
    import oracle.build as O
    from weight_only_quantized_msd_amd import build as B
    done = []
    monkeypatch.setattr(B, "build", lambda *a: done.append("library"))
    monkeypatch.setattr(B, "build_calls", lambda *a: done.append("calls"))
    monkeypatch.setattr(O, "build", lambda *a: done.append("oracle"))
    return entry, done


def test_with_torch(steps):
    entry, done = steps
    pytest.importorskip("torch")
    entry.build()
    assert done == ["library", "oracle", "calls"]


def test_without_torch(steps, monkeypatch, capsys):
    entry, done = steps
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch raises ImportError
    entry.build()
    assert done == ["library", "oracle"] and "no torch" in capsys.readouterr().out
