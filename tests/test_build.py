"""What build() builds and when, with a compiler that only writes its output file."""
import importlib.util
import os
import stat
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMPILER = """#!/bin/sh
echo "$@" >> "$(dirname "$0")/calls"
while [ $# -gt 0 ]; do [ "$1" = "-o" ] && echo built > "$2"; shift; done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build.py on its own, as a script has it, building into a folder of its own."""
    spec = importlib.util.spec_from_file_location("build_alone", os.path.join(HERE, "rope_block_sparse_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    for name in ("nvcc", "g++"):
        (tmp_path / name).write_text(COMPILER)
        (tmp_path / name).chmod(stat.S_IRWXU)
    monkeypatch.setenv("PATH", f"{tmp_path}{os.pathsep}{os.environ['PATH']}")
    build.BUILD, build.PKG = str(tmp_path / "_build"), str(tmp_path)
    build.LIB = str(tmp_path / "libh3a.so")
    build.calls = lambda: (tmp_path / "calls").read_text().splitlines() if (tmp_path / "calls").exists() else []
    return build


@pytest.mark.parametrize("installed", ["none", "without CUDA"])
def test_the_library_needs_no_torch(tree, monkeypatch, capsys, installed):
    if installed == "none":
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch: ModuleNotFoundError
    else:
        monkeypatch.setattr(torch.version, "cuda", None)
    assert tree.needs_build()
    assert tree.build() == tree.LIB
    assert os.path.exists(tree.LIB) and len(tree.calls()) == len(tree.SOURCES) + 1
    assert not tree.needs_build()
    assert "binding is not" in capsys.readouterr().err


def test_both_are_built_once(tree):
    assert tree.needs_build()
    tree.build()
    binding = tree.binding_path(torch)
    assert os.path.exists(tree.LIB) and os.path.exists(binding)
    assert len(tree.calls()) == len(tree.SOURCES) + 2 and not tree.needs_build()
    tree.build()
    assert len(tree.calls()) == len(tree.SOURCES) + 2
    os.remove(binding)
    assert tree.needs_build()
    tree.build()
    assert "binding.cpp" in tree.calls()[-1] and len(tree.calls()) == len(tree.SOURCES) + 3
    tree.build(force=True)
    assert len(tree.calls()) == 2 * len(tree.SOURCES) + 5


@pytest.mark.parametrize("what", ["torch", "C++ ABI", "Python"])
def test_another_torch_or_python_gets_a_binding_of_its_own(tree, monkeypatch, what):
    tree.build()
    before = tree.binding_path(torch)
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    elif what == "C++ ABI":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-999")
    assert tree.needs_build()
    tree.build()
    assert "binding.cpp" in tree.calls()[-1] and len(tree.calls()) == len(tree.SOURCES) + 3
    assert tree.binding_path(torch) != before and os.path.exists(tree.binding_path(torch)) and not tree.needs_build()


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    from rope_block_sparse_b200 import h3a

    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    with pytest.raises(RuntimeError, match="build it for this torch"):
        h3a._binding.__wrapped__()
