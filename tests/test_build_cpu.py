"""The build of the library and of the torch binding (no GPU)."""
import os

import pytest

from context_varlen_ring_gb300 import build as b


@pytest.fixture
def apart(monkeypatch, tmp_path):
    """The library and the binding linked into a folder of their own, from the objects at hand."""
    b.build()
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libra.so"))
    monkeypatch.setattr(b, "MODULE", str(tmp_path / "_serving.so"), raising=False)
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
