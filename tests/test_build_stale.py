"""When the marshalling module is built anew (no GPU)."""
import os

import pytest
import torch

from gated_delta_rule_08_gb300 import build


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A module that has just been built from one source."""
    source, module, mark = tmp_path / "a.cpp", tmp_path / "a.so", tmp_path / "mark"
    for f in (source, module):
        f.write_text("")
    mark.write_text(build._marshal_for())
    monkeypatch.setattr(build, "MARSHAL", str(module))
    monkeypatch.setattr(build, "MARSHAL_FOR", str(mark))
    os.utime(source, (1, 1))
    return source, module, mark


def test_a_module_is_kept(built):
    assert not build._marshal_stale([str(built[0])])


def test_a_changed_source_or_no_module(built):
    source, module, _ = built
    os.utime(source, (2 ** 31, 2 ** 31))
    assert build._marshal_stale([str(source)])
    os.utime(source, (1, 1))
    module.unlink()
    assert build._marshal_stale([str(source)])


def test_another_torch(built, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert build._marshal_stale([str(built[0])])


def test_no_record_of_what_it_was_built_against(built):
    built[2].unlink()
    assert build._marshal_stale([str(built[0])])
