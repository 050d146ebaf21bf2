"""The library is built without what only the Python binding needs (a host compiler of its own, Python's and torch's
headers); a binding is out of date when it was built for another torch."""
import os
import subprocess

import pytest

import fp8_moe_expert_gb300 as fme
from fp8_moe_expert_gb300 import build as fme_build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A package whose library is one empty translation unit."""
    src = tmp_path / "empty.cu"
    src.write_text("extern \"C\" int fme_empty() { return 0; }\n")
    monkeypatch.setattr(fme_build, "SOURCES", [str(src)])
    monkeypatch.setattr(fme_build, "HEADERS", [])
    monkeypatch.setattr(fme_build, "LIBRARY", str(tmp_path / "libsmall.so"))
    monkeypatch.setattr(fme_build, "BINDING", str(tmp_path / "_small.so"))
    return fme_build


def test_library_without_a_binding(small, monkeypatch):
    monkeypatch.setenv("CXX", "false")  # a compiler that always fails
    with open(small.BINDING, "w") as f:
        f.write("an outdated one")
    with pytest.warns(RuntimeWarning, match="binding was not built"):
        small.build(output=small.LIBRARY)
    out = subprocess.run(["nm", "-D", small.LIBRARY], capture_output=True, text=True, check=True).stdout
    assert "fme_empty" in out and not os.path.exists(small.BINDING)


def test_missing_compiler_leaves_the_library_alone(small, monkeypatch):
    monkeypatch.setenv("CXX", "/nonexistent/c++")
    with pytest.warns(RuntimeWarning, match="binding was not built"):
        small.build(output=small.LIBRARY)
    built = os.path.getmtime(small.LIBRARY)
    with pytest.warns(RuntimeWarning, match="binding was not built"):
        small.refresh()  # tries the binding again, not the library
    assert os.path.getmtime(small.LIBRARY) == built


def test_a_library_that_fails_still_raises(small, monkeypatch, tmp_path):
    bad = tmp_path / "bad.cu"
    bad.write_text("not C++\n")
    monkeypatch.setattr(small, "SOURCES", [str(bad)])
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        small.build(output=small.LIBRARY)


def test_binding_for_another_torch(monkeypatch):
    torch = pytest.importorskip("torch")
    fme.ensure_built()
    assert not fme_build.stale()
    monkeypatch.setattr(torch, "__version__", "99.9.0")
    assert fme_build.stale()
    monkeypatch.setattr(fme, "_native", None)
    with pytest.raises(RuntimeError, match="built for torch .*, this is torch 99.9.0"):
        fme._bind()
