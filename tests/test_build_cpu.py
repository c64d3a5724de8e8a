"""What a build makes without torch, when the binding's module fails to compile, and after Python or torch changed."""
import importlib.machinery
import importlib.metadata
import importlib.util
import os

import pytest

from kronecker_sparse_matrix_b200 import build as ksbuild


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The products' places in a folder of the test's own; the compiled objects are the real ones."""
    ksbuild.build()
    monkeypatch.setattr(ksbuild, "LIB", str(tmp_path / "libks_b200.so"))
    monkeypatch.setattr(ksbuild, "MARSHAL", str(tmp_path / os.path.basename(ksbuild.MARSHAL)))
    monkeypatch.setattr(ksbuild, "MARSHAL_STAMP", str(tmp_path / "stamp"), raising=False)
    return tmp_path


def test_the_library_is_built_without_torch(elsewhere, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert ksbuild.build() == ksbuild.LIB and os.path.exists(ksbuild.LIB)
    assert not os.path.exists(ksbuild.MARSHAL)


def test_the_library_is_built_where_the_module_does_not_compile(elsewhere, monkeypatch):
    broken = elsewhere / "ks_marshal.cpp"
    broken.write_text("#error no DLPack exchange functions\n")
    monkeypatch.setattr(ksbuild, "MARSHAL_SRC", str(broken))
    with pytest.raises(RuntimeError, match="ks_marshal"):
        ksbuild.build()
    assert os.path.exists(ksbuild.LIB) and not os.path.exists(ksbuild.MARSHAL)


def test_the_module_follows_python_and_torch(elsewhere, monkeypatch):
    assert ksbuild.MARSHAL.endswith(importlib.machinery.EXTENSION_SUFFIXES[0])
    ksbuild.build_marshal()
    first = os.stat(ksbuild.MARSHAL).st_mtime_ns, os.stat(ksbuild.MARSHAL).st_ino

    def now():
        ksbuild.build_marshal()
        return os.stat(ksbuild.MARSHAL).st_mtime_ns, os.stat(ksbuild.MARSHAL).st_ino

    assert now() == first
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0" if name == "torch" else version(name))
    second = now()
    assert second != first and now() == second
