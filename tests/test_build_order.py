"""The build makes the C library whatever becomes of the Python module beside
it (CPU; no compiler is run)."""

import os

import pytest

from memory_bound_w8a8_amd import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    for name in ("LIB", "BINDING"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "_hipcc", lambda: "hipcc")
    (tmp_path / "_binding.so").write_text("of an earlier build")
    return tmp_path


def _writes(fails=None):
    def run(cmd):
        if fails and any(fails in word for word in cmd):
            raise RuntimeError("command failed")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return ""

    return run


def test_both_are_built(tree, monkeypatch):
    monkeypatch.setattr(build, "_run", _writes())
    assert build.build() == build.LIB
    assert (tree / "libfp8bq.so").read_text() == (tree / "_binding.so").read_text() == "built"


@pytest.mark.parametrize("fails", ["binding.cpp", "-ltorch_python"])
def test_library_is_there_where_the_module_cannot_be_built(tree, monkeypatch, fails):
    monkeypatch.setattr(build, "_run", _writes(fails))
    with pytest.raises(RuntimeError):  # it is said all the same
        build.build()
    assert (tree / "libfp8bq.so").read_text() == "built"
    assert not (tree / "_binding.so").exists()  # none that an older library was built with


def test_library_is_there_without_torchs_headers(tree, monkeypatch):
    def no_torch(obj):
        raise ImportError("no torch headers")

    monkeypatch.setattr(build, "_run", _writes())
    monkeypatch.setattr(build, "_binding_compile", no_torch)
    with pytest.raises(ImportError):
        build.build()
    assert (tree / "libfp8bq.so").read_text() == "built"


def test_a_kernel_that_does_not_compile_leaves_the_library(tree, monkeypatch):
    (tree / "libfp8bq.so").write_text("of an earlier build")
    monkeypatch.setattr(build, "_run", _writes("verify.hip"))
    with pytest.raises(RuntimeError):
        build.build()
    assert (tree / "libfp8bq.so").read_text() == "of an earlier build"
