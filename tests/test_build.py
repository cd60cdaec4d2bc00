"""The library needs no Python or torch headers, and the binding is rebuilt for
another torch or Python."""
import os

import pytest

import gated_deltanet_paged_gb300 as gdn
from gated_deltanet_paged_gb300 import build


def _no_torch():
    raise RuntimeError("no headers")


def test_library_is_built_where_the_binding_cannot_be(monkeypatch, tmp_path):
    gdn.library()
    monkeypatch.setattr(build, "_torch_paths", _no_torch)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_attention.so"))
    assert build.up_to_date() and not build.binding_up_to_date()
    assert build.build_library() == build.LIB
    built = []
    monkeypatch.setattr(build, "build_library", lambda *a: built.append(a) or build.LIB)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert built, "the library waits for nothing that the binding needs"
    with pytest.raises(RuntimeError, match="no headers"):
        build.build_binding()


def test_library_does_not_wait_for_the_binding(monkeypatch, tmp_path):
    """Loading the library for the recurrent layer's calls asks for no binding."""
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_attention.so"))
    monkeypatch.setattr(build, "build_binding", lambda *a: pytest.fail("the binding was built"))
    monkeypatch.setattr(gdn, "_lib", None)
    gdn.library()


def test_binding_of_another_torch_or_python_is_out_of_date(monkeypatch, tmp_path):
    build.build_binding()
    assert build.binding_up_to_date()
    key = build._binding_key()
    for what in ("another " + key, ""):
        other = tmp_path / "binding.txt"
        other.write_text(what)
        monkeypatch.setattr(build, "BINDING_KEY", str(other))
        assert not build.binding_up_to_date()
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "none"))
    assert not build.binding_up_to_date()
    monkeypatch.undo()
    assert build.binding_up_to_date() and os.path.exists(build.BINDING)
