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
