"""The build of the library and of the torch binding (no GPU)."""
import os

import pytest
import torch

from context_varlen_ring_gb300 import build as b


@pytest.fixture
def apart(monkeypatch, tmp_path):
    """The library and the binding linked into a folder of their own, from the objects at hand."""
    b.build()
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libra.so"))
    monkeypatch.setattr(b, "module_path", lambda: str(tmp_path / "_serving.so"), raising=False)
    return tmp_path


@pytest.mark.parametrize("why", ["source", "torch"])
def test_the_library_is_built_without_the_binding(apart, monkeypatch, capsys, why):
    """A binding that does not compile, or no torch to compile it for: the library is linked all the same, what was there
    of an older binding is gone, and the reason is told."""
    (apart / "_serving.so").write_bytes(b"old")
    if why == "source":
        (apart / "broken.cpp").write_text("#error no such torch\n")
        monkeypatch.setattr(b, "MODULE_SRC", str(apart / "broken.cpp"))
    else:
        def gone(*a, **k):
            raise ImportError("no such torch")
        monkeypatch.setattr(b, "_module_job", gone)
    assert b.build() == str(apart / "libra.so")
    assert os.path.getsize(apart / "libra.so") > 0 and not (apart / "_serving.so").exists()
    assert "no such torch" in capsys.readouterr().err


def test_each_environment_has_a_binding_of_its_own(monkeypatch):
    """Built for one torch, then another, then called again under the first: the first one's file is still its own."""
    b.build()
    import context_varlen_ring_gb300 as ra
    here = b.module_path()
    assert ra.serving._native().__file__ == here and ra.serving._native().rope
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert b.module_path() != here and not os.path.exists(b.module_path())
    monkeypatch.setattr(ra.serving, "_mod", None)
    with pytest.raises(ImportError):
        ra.serving._native()
