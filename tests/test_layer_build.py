"""The command that builds the library, where there is a torch to bind to and where there is none."""
import sys

import pytest

from tensor_core_tiled_02_gb300 import build as tcbuild


@pytest.mark.parametrize("argv,variant", [([], ""), (["trace"], "trace"), (["-v", "check"], "check")])
def test_library_without_torch(monkeypatch, capsys, argv, variant):
    """The library comes first and does not need torch; the binding is left out, and it is said."""
    built = []
    monkeypatch.setattr(tcbuild, "build", lambda verbose_ptxas=False, variant="": built.append((variant, verbose_ptxas)) or "lib")
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises
    tcbuild.main(argv)
    assert built == [(variant, "-v" in argv)]
    assert "no torch binding" in capsys.readouterr().out


def test_library_first(monkeypatch):
    built = []
    monkeypatch.setattr(tcbuild, "build", lambda **k: built.append("library") or "lib")
    monkeypatch.setattr(tcbuild, "build_binding", lambda: built.append("binding") or "binding")
    tcbuild.main([])
    assert built == ["library", "binding"]
