"""What the build makes, and from what, with the compilers replaced by a
recorder that leaves an empty output file."""
import importlib.machinery
import importlib.util
import os

import pytest

from sparse_selected_attention_gb300 import build


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The outputs of the commands that ran, in order; all files in a folder of the test's own."""
    names = []

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        names.append(os.path.basename(out).removesuffix(".tmp"))

        class Result:
            stdout = stderr = ""
        return Result
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_paged_binding.so"))
    monkeypatch.setattr(build, "_run", run)
    return names


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_builds_without_torch(made, tmp_path, monkeypatch):
    without_torch(monkeypatch)
    lib = build.build()
    assert os.path.exists(lib) and made[-1] == "libqsa.so" and "_paged_binding.so" not in made
    assert not (tmp_path / "_paged_binding.so").exists()


def test_the_library_builds_beside_a_torch_without_cuda(made, tmp_path, monkeypatch):
    spec = importlib.machinery.ModuleSpec("torch", None, origin=str(tmp_path / "torch" / "__init__.py"))
    (tmp_path / "torch" / "lib").mkdir(parents=True)
    (tmp_path / "torch" / "version.py").write_text("__version__ = '2.9.0+cpu'")
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    assert os.path.exists(build.build()) and "_paged_binding.so" not in made


def test_a_binding_that_does_not_build_leaves_the_library(made, tmp_path, monkeypatch):
    def broken(*args):
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "build_binding", broken)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert (tmp_path / "libqsa.so").exists()


def test_the_library_and_its_binding(made, tmp_path):
    build.build()
    assert sorted(made) == sorted([s + ".o" for s in build.SOURCES] + ["libqsa.so", "_paged_binding.so"])
    made.clear()
    build.build()
    assert made == []
    build.build(variant="check")
    assert "_paged_binding.so" not in made and made[-1] == "libqsa_check.so"


# ---------------------------------------------------------------- the binding's torch

def test_a_binding_of_another_torch_is_rebuilt(made, tmp_path, monkeypatch):
    build.build()
    made.clear()
    for name in ("torch_version", "abi_tag"):
        with monkeypatch.context() as m:
            m.setattr(build, name, lambda: "another")
            build.build()
            assert made == ["_paged_binding.so"], name
            build.build()
            assert made == ["_paged_binding.so"], name
        made.clear()
        build.build()
        assert made == ["_paged_binding.so"], name  # and back
        made.clear()
    os.remove(build.binding_stamp())  # a file whose torch is not known
    build.build()
    assert made == ["_paged_binding.so"]


def test_what_is_compiled_in_is_what_is_loaded():
    import torch
    build.build()
    from sparse_selected_attention_gb300 import _paged_binding, paged
    assert _paged_binding.torch_version == torch.__version__ == build.torch_version()
    assert _paged_binding.abi_tag == build.abi_tag()
    assert paged.binding_of_this_torch() is _paged_binding


@pytest.mark.parametrize("name", ["torch_version", "abi_tag"])
def test_a_binding_of_another_torch_is_refused(monkeypatch, name):
    build.build()
    from sparse_selected_attention_gb300 import _paged_binding, paged
    monkeypatch.setattr(_paged_binding, name, "1.2.3")
    with pytest.raises(RuntimeError, match="1.2.3.*sparse_selected_attention_gb300.build"):
        paged.binding_of_this_torch()
