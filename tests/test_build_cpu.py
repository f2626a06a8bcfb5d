"""The build where the compiled checks of the binding cannot be made: the library is built all the same."""
import importlib.metadata
import os
import sys

import pytest

from activation_epilogue_tcgen05_b200 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """build_operands() into an empty folder, from the same source."""
    monkeypatch.setattr(build, "OPERANDS_SO", str(tmp_path / "_operands.so"))
    return tmp_path


@pytest.mark.parametrize("cxx", ["/nowhere/c++", "false", os.path.dirname(os.path.abspath(__file__))])
def test_without_a_compiler(elsewhere, monkeypatch, capsys, cxx):
    monkeypatch.setenv("CXX", cxx)
    (elsewhere / "_operands.so").write_bytes(b"of another source")
    assert build.build_operands() is False
    assert "checks its operands in Python" in capsys.readouterr().err and not list(elsewhere.iterdir())


def test_without_torch(elsewhere, monkeypatch, capsys):
    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(importlib.metadata, "version", missing)
    monkeypatch.setitem(sys.modules, "torch", None)           # (an import of it is an ImportError)
    assert build.build_operands() is False
    assert "checks its operands in Python" in capsys.readouterr().err


def test_into_a_folder_that_cannot_be_written(tmp_path, monkeypatch, capsys):
    monkeypatch.setattr(build, "OPERANDS_SO", str(tmp_path / "missing" / "_operands.so"))
    assert build.build_operands() is False
    assert "checks its operands in Python" in capsys.readouterr().err
