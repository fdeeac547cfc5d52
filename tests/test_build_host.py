"""The build without a GPU or a compiler run: what the library and the binding's
extension each need, and what the binding says when the extension does not load."""
from __future__ import annotations

import subprocess
import sys
from pathlib import Path

import pytest

from gated_delta_rule_40_amd import build

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture
def bare(tmp_path, monkeypatch):
    """A build of no sources whose linker only writes its output file."""
    linker = tmp_path / "linker"
    linker.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho linked > "$2"\n')
    linker.chmod(0o755)
    monkeypatch.setenv("HIPCC", str(linker))
    monkeypatch.setattr(build, "sources", lambda: [])
    monkeypatch.setattr(build, "BUILD_DIR", tmp_path / "objects")
    monkeypatch.setattr(build, "LIB_PATH", tmp_path / "lib.so")
    monkeypatch.setattr(build, "MARSHAL_PATH", tmp_path / "_marshal.so")
    return tmp_path


@pytest.mark.parametrize("lacking", ["torch", "Python.h"])
def test_library_links_without_what_only_the_extension_needs(bare, monkeypatch, capsys, lacking):
    if lacking == "torch":
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(bare)})
    assert build.build_library(jobs=1) == bare / "lib.so"
    assert (bare / "lib.so").read_text() == "linked\n" and not (bare / "_marshal.so").exists()
    assert f"no {lacking}" in capsys.readouterr().err


def test_library_is_in_place_when_the_extension_fails(bare, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="_marshal.so failed"):
        build.build_library(jobs=1)
    assert (bare / "lib.so").exists()


def test_binding_says_why_the_extension_does_not_load():
    code = """
import sys
sys.modules["gated_delta_rule_40_amd._marshal"] = None
from gated_delta_rule_40_amd import binding
try:
    binding._ptr(None)
except RuntimeError as e:
    print(e, "|", type(e.__cause__).__name__)
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert "cannot be loaded (import of gated_delta_rule_40_amd._marshal halted" in out.stdout
    assert "| ModuleNotFoundError" in out.stdout or "| ImportError" in out.stdout
