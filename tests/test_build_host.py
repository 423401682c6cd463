"""When the build makes what (no compiler is run here)."""
import os

import pytest

from vision_test_token_b200 import build as b


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Fresh outputs in a folder of their own, and the list of what the build makes."""
    made = []
    for name in ("OUT", "NATIVE", "NATIVE_KEY"):
        monkeypatch.setattr(b, name, str(tmp_path / name))

    def touch(what, path):
        made.append(what)
        open(path, "w").close()

    monkeypatch.setattr(b, "_build_lib", lambda verbose: touch("lib", b.OUT))
    monkeypatch.setattr(b, "_build_native", lambda: touch("native", b.NATIVE))
    monkeypatch.setattr(b, "_native_key", lambda: "torch 1")
    assert b.build() == b.OUT and made == ["lib", "native"]
    made.clear()
    return made


def test_nothing_twice(made):
    b.build()
    assert made == []
    b.build(force=True)
    assert made == ["lib", "native"]


def test_another_torch_makes_the_binding_again(made, monkeypatch):
    monkeypatch.setattr(b, "_native_key", lambda: "torch 2")
    b.build()
    b.build()
    assert made == ["native"]


def test_without_torch_the_library_is_built(made, monkeypatch, capsys):
    monkeypatch.setattr(b, "_native_key", lambda: None)
    os.remove(b.OUT)
    assert b.build() == b.OUT and made == ["lib"]
    assert "no torch" in capsys.readouterr().err


def test_sources_decide(made, monkeypatch, tmp_path):
    later = os.path.getmtime(b.OUT) + 100
    source = tmp_path / "kernel.cu"
    source.write_text("")
    os.utime(source, (later, later))
    monkeypatch.setattr(b, "_lib_deps", lambda: [str(source)])
    b.build()
    assert made == ["lib"]                        # the binding's sources are as they were


def test_key_names_torch():
    import torch
    assert torch.__version__.split("+")[0] in b._native_key()
