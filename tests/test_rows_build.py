"""The build of the library does not depend on the row operators' Python
binding, and a binding made for another PyTorch is not used. Host only; the
compilers are stood in for."""
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


def test_a_binding_for_another_torch_does_not_count(monkeypatch):
    _build.build()
    assert _build.binding_up_to_date()
    here = _build.binding_path()
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert _build.binding_path() != here and not _build.binding_up_to_date()


def test_a_binding_made_before_its_flags_changed_does_not_count(monkeypatch, tmp_path):
    path = tmp_path / "binding.so"
    path.write_bytes(b"")
    monkeypatch.setattr(_build, "binding_path", lambda: str(path))
    newest = max(os.path.getmtime(f) for f in (_build.__file__, _build.BINDING_SRC))
    os.utime(path, (newest + 1, newest + 1))
    assert _build.binding_up_to_date()
    before = os.path.getmtime(_build.__file__) - 1
    os.utime(path, (before, before))
    assert not _build.binding_up_to_date()
