"""When build.py compiles the binding's compiled part again (the compiler is replaced by a stand-in)."""

import os

import pytest

from w4a8_codebook_quantized_rotate_b200 import build as W


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The list of compilations, which leave an empty file."""
    runs = []

    def run(cmd, check):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(W.subprocess, "run", run)
    monkeypatch.setattr(W, "MARSHAL_OUT", str(tmp_path / "marshal.so"))
    if hasattr(W, "MARSHAL_AGAINST"):
        monkeypatch.setattr(W, "MARSHAL_AGAINST", str(tmp_path / "marshal.so.against"))
    return runs


def test_compiled_once_for_its_sources_and_torch(compiled, monkeypatch, tmp_path):
    import torch
    W.build_marshal()
    W.build_marshal()
    assert len(compiled) == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "x")       # another torch in its place
    W.build_marshal()
    W.build_marshal()
    assert len(compiled) == 2
    monkeypatch.undo()


def test_compiled_again_for_newer_sources_or_without_a_record(compiled, tmp_path):
    W.build_marshal()
    os.utime(W.MARSHAL_OUT, (0, 0))
    W.build_marshal()
    assert len(compiled) == 2
    os.remove(W.MARSHAL_AGAINST)
    W.build_marshal()
    W.build_marshal()
    assert len(compiled) == 3
    W.build_marshal(force=True)
    assert len(compiled) == 4
