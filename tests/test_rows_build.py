"""The build of the library does not depend on the row operators' Python
binding. Host only; the compilers are stood in for."""
import os

import pytest
import torch

from segmented_radix_top_gb300 import _build, _rows


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Nothing is up to date; a list of what is compiled and linked."""
    done = []
    monkeypatch.setattr(_build, "VARIANTS", {"": (str(tmp_path / "objects"), str(tmp_path / "lib.so"), [])})
    monkeypatch.setattr(_build, "binding_path", lambda: str(tmp_path / "binding.so"), raising=False)
    monkeypatch.setattr(_build, "_compile", lambda variant, src, flags, verbose: src)
    monkeypatch.setattr(_build, "_link", lambda variant, objs: done.append(("library", len(objs))))
    monkeypatch.setattr(_build, "_compile_binding", lambda verbose: done.append("binding"))
    return done


def test_the_library_is_linked_where_the_binding_does_not_compile(made, monkeypatch):
    def fails(verbose):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(_build, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        _build.build(force=True)
    assert made == [("library", len(_build._sources()))]


def test_the_library_is_built_alone_without_the_headers(made, monkeypatch, capfd):
    monkeypatch.setattr(_build, "_binding_includes", lambda: [os.path.join(os.sep, "nowhere")], raising=False)
    _build.build(force=True)
    assert made == [("library", len(_build._sources()))]
    assert "Python.h" in capfd.readouterr().err
    monkeypatch.setattr(_rows, "_native", None)
    monkeypatch.setattr(_rows.B, "load", lambda: None)
    with pytest.raises(RuntimeError, match="Python.h"):
        _rows.route(torch.zeros(1, 1), 1)


def test_both_are_built_where_both_can_be(made):
    assert _build.binding_lacks() == []
    _build.build(force=True)
    assert sorted(made, key=str) == sorted([("library", len(_build._sources())), "binding"], key=str)
