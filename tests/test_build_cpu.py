"""The build's two parts: the CUDA library needs no torch, the binding is built for one."""
import sys

import pytest

from selective_state_space_27_b200 import build as msbuild


@pytest.fixture
def recorded(monkeypatch):
    """The parts that build() compiles, without compiling them."""
    made = []
    monkeypatch.setattr(msbuild, "build_library", lambda *a: made.append("library") or msbuild.LIB)
    monkeypatch.setattr(msbuild, "build_binding", lambda *a: made.append("binding") or msbuild.BINDING)
    return made


def test_library_is_built_without_torch(recorded, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)   # (import torch raises ModuleNotFoundError)
    assert msbuild.build(force=True) == msbuild.LIB
    assert recorded == ["library"] and "torch is not installed" in capsys.readouterr().out


def test_both_parts_are_built(recorded):
    assert msbuild.build(force=True) == msbuild.LIB
    assert recorded == ["library", "binding"]


def test_binding_is_rebuilt_for_another_torch(recorded, monkeypatch, tmp_path):
    """The files are as old as they were, the torch or the Python is another one."""
    import torch
    for name in ("BINDING", "BINDING_FOR"):
        monkeypatch.setattr(msbuild, name, str(tmp_path / name))
    monkeypatch.setattr(msbuild, "up_to_date", lambda: True)
    (tmp_path / "BINDING").write_text("")
    (tmp_path / "BINDING_FOR").write_text(msbuild._interpreter())
    msbuild.build()
    assert recorded == [] and msbuild.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    msbuild.build()
    assert recorded == ["binding"]
    (tmp_path / "BINDING_FOR").unlink()
    msbuild.build()
    assert recorded == ["binding"] * 2
