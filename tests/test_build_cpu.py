"""The in-tree build: what it compiles and when it does so again (commands are recorded, not run)."""
import os

import pytest

from paged_kv_cache_295_gb300 import _build


@pytest.fixture
def recorded(tmp_path, monkeypatch):
    """The build with its outputs under ``tmp_path`` and its commands only recorded."""
    for name, f in (("LIB", "libpagedkv.so"), ("BINDING", "_pkv_torch.so"), ("BUILD", "_build")):
        monkeypatch.setattr(_build, name, str(tmp_path / f))
    commands = []

    def run(cmd):
        commands.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w"):
            pass
        return ""
    monkeypatch.setattr(_build, "_run", run)
    return commands


def test_library_builds_without_torch(recorded, monkeypatch):
    """The C ABI needs no torch: without it the library is compiled and linked and the binding
    left out."""
    monkeypatch.setitem(__import__("sys").modules, "torch", None)      # as not installed
    assert _build.build_library() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING)
    assert not any(part.startswith("-ltorch") or "torch_binding" in part for cmd in recorded for part in cmd)
    assert not _build.stale()


def test_binding_builds_with_torch(recorded):
    pytest.importorskip("torch")
    _build.build_library()
    assert os.path.exists(_build.LIB) and os.path.exists(_build.BINDING)
    links = [cmd for cmd in recorded if "-shared" in cmd]
    assert len(links) == 2 and "-ltorch_python" not in links[0] and "-ltorch_python" in links[1]
    assert not _build.stale()
    del recorded[:]
    _build.build_library()
    assert not recorded


def test_another_torch_or_python_rebuilds_the_binding(recorded, monkeypatch):
    pytest.importorskip("torch")
    _build.build_library()
    monkeypatch.setattr(_build.importlib.metadata, "version", lambda name: "99.0")
    assert _build.stale()
    del recorded[:]
    _build.build_library()
    assert any("-ltorch_python" in cmd for cmd in recorded) and not _build.stale()


def test_binding_of_another_torch_is_not_loaded(recorded, monkeypatch, lib):
    pytest.importorskip("torch")
    _build.build_library()
    monkeypatch.setattr(lib, "_ext", None)
    monkeypatch.setattr(_build.importlib.metadata, "version", lambda name: "99.0")
    with pytest.raises(RuntimeError, match="built for torch"):
        lib._binding()
