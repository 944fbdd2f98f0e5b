"""What the two built files depend on: the extension on the torch and the Python that it was
built with, the library on neither."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT
from serving_lightning_indexer_gb300 import _build, csa2


def test_an_extension_of_another_torch_is_not_loaded_and_built_again(monkeypatch):
    _build.build()
    assert _build.call_made_with() == _build.made_with()
    ran = []
    monkeypatch.setattr(_build, "made_with", lambda: "cpython-399, torch 99.0")
    monkeypatch.setattr(_build, "_compile_call", lambda verbose: ran.append("compile") or "binding.o")
    monkeypatch.setattr(_build, "_link_call", lambda obj, verbose: ran.append("link " + obj))
    with pytest.raises(RuntimeError, match="built with cpython.* this is cpython-399, torch 99.0"):
        csa2._load_call()
    _build.build()
    assert ran == ["compile", "link binding.o"]


def test_an_extension_that_does_not_say_is_built_again(monkeypatch, tmp_path):
    _build.build()
    monkeypatch.setattr(_build, "CALL_MADE_WITH", str(tmp_path / "none"))
    ran = []
    monkeypatch.setattr(_build, "_compile_call", lambda verbose: ran.append("compile") or "binding.o")
    monkeypatch.setattr(_build, "_link_call", lambda obj, verbose: ran.append("link"))
    _build.build()
    assert ran == ["compile", "link"]


def test_the_library_builds_without_torch():
    code = ("import sys; sys.modules['torch'] = None\n"
            "from serving_lightning_indexer_gb300 import _build\n"
            "print(_build.build_library())\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert os.path.exists(r.stdout.strip())
