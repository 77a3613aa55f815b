"""What the build does with its two products, the compilers replaced by
functions that write empty files."""
import os

import pytest

from sparse_mla_decode_dcp_gb300 import build as smla_build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build in a folder of its own; returns the products made, in order."""
    made = []

    def touch(path):
        with open(path, "w"):
            pass
        made.append(os.path.basename(path))
        return path

    monkeypatch.setattr(smla_build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(smla_build, "LIB_PATH", str(tmp_path / "libsmla.so"))
    monkeypatch.setattr(smla_build, "BINDING_PATH", str(tmp_path / "_smla_torch.so"))
    monkeypatch.setattr(smla_build, "_compile", lambda nvcc, src, obj, log_dir: touch(obj))
    monkeypatch.setattr(smla_build, "_compile_binding", lambda obj, log_dir: touch(obj))
    monkeypatch.setattr(smla_build, "_link", lambda cmd: touch(cmd[cmd.index("-o") + 1]))
    return made


def test_a_second_build_makes_nothing(tree):
    smla_build.build()
    assert {"libsmla.so", "_smla_torch.so", "smla_torch.o"} <= set(tree)
    del tree[:]
    smla_build.build()
    assert tree == []


def test_the_library_is_linked_when_the_binding_does_not_compile(tree, monkeypatch):
    def fails(obj, log_dir):
        raise RuntimeError("the binding failed to compile")

    with monkeypatch.context() as m:
        m.setattr(smla_build, "_compile_binding", fails)
        with pytest.raises(RuntimeError, match="binding"):  # not in silence
            smla_build.build()
    assert "libsmla.so" in tree and "_smla_torch.so" not in tree
    smla_build.build()  # and the binding follows once it does
    assert "_smla_torch.so" in tree


def test_the_binding_follows_the_installed_torch(tree, monkeypatch):
    smla_build.build()
    del tree[:]
    key = smla_build._torch_key()
    monkeypatch.setattr(smla_build, "_torch_key", lambda: key + "another version")
    smla_build.build()
    assert tree == ["smla_torch.o", "_smla_torch.so"]  # the library stays


def test_the_library_needs_no_torch(tree, monkeypatch):
    import importlib.util
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    smla_build.build()
    assert "libsmla.so" in tree and "_smla_torch.so" not in tree
