"""What build() builds, with the compilers replaced by ones that only make their output files."""
import os
import sys
import types

import pytest

from sparse_attention_indexer_tiles_gb300 import build as b


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """The names of the files that each build makes."""
    made = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(os.path.basename(out).split(".")[0])
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libidx.so"))
    monkeypatch.setattr(b, "BINDING_LIB", str(tmp_path / "_serve.so"))

    def build():
        made.clear()
        lib = b.build()
        assert lib == str(tmp_path / "libidx.so") and os.path.exists(lib)
        return set(made)

    return types.SimpleNamespace(build=build, path=tmp_path)


OBJECTS = {os.path.basename(s)[:-3] for s in b.sources()}


def test_all_of_it_once(tree):
    assert tree.build() == OBJECTS | {"libidx", "_serve"}
    assert tree.build() == set()


def test_the_c_library_needs_no_pytorch(monkeypatch, tree):
    import importlib.metadata

    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(importlib.metadata, "version", missing)
    assert tree.build() == OBJECTS | {"libidx"}
    assert not (tree.path / "_serve.so").exists()
    assert tree.build() == set()


def test_another_pytorch_needs_another_binding(monkeypatch, tree):
    import importlib.metadata
    tree.build()
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0")
    assert tree.build() == {"_serve"}
    assert tree.build() == set()


def test_a_binding_that_does_not_build_leaves_the_library(monkeypatch, tree):
    run = b.subprocess.run

    def no_host_compiler(cmd, **kw):
        if b.BINDING in cmd:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="")
        return run(cmd, **kw)

    monkeypatch.setattr(b.subprocess, "run", no_host_compiler)
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert (tree.path / "libidx.so").exists() and not (tree.path / "_serve.so").exists()


def test_a_changed_source_is_built_again(tree):
    tree.build()
    for name, what in (("libidx.so", OBJECTS | {"libidx"}), ("_serve.so", {"_serve"})):
        os.utime(tree.path / name, (1, 1))
        assert tree.build() == what
