"""What the build makes again and when: the CUDA library by its sources alone, the extension for the torch and Python
that it is bound to. In a folder of its own, the compilers replaced by a record of their calls."""

import os
import subprocess
import types

import pytest
import torch

from top_gating_expert_gb300 import build as b


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The names of what was compiled or linked, in order; `made.fails`: a compiler that reports an error."""
    made = types.SimpleNamespace(names=[], fails=None)

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        tool = os.path.basename(cmd[0])
        if tool == made.fails:
            return subprocess.CompletedProcess(cmd, 1, "", "no headers")
        made.names.append(os.path.basename(out))
        with open(out, "w") as f:
            f.write("x")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "PKG", str(tmp_path))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "_nvcc", lambda: "/x/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.delenv("CXX", raising=False)
    return made


def test_each_part_by_itself(made, monkeypatch):
    b.build_library()
    assert "_lists.so.tmp" in made.names and "libmoe_gb300.so.tmp" in made.names and "xent.o" in made.names
    assert os.path.exists(b.library_path()) and os.path.exists(b.lists_path())
    made.names.clear()
    b.build_library()
    assert made.names == []
    for change in (lambda: monkeypatch.setattr(torch, "__version__", "9.9.0"),
                   lambda: monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399"),
                   lambda: os.remove(b.lists_path()), lambda: os.remove(b._lists_stamp())):
        change()
        b.build_library()
        assert made.names == ["_lists.so.tmp"]
        made.names.clear()
        b.build_library()
        assert made.names == []
    os.remove(b.library_path())
    b.build_library()
    assert "_lists.so.tmp" not in made.names and "libmoe_gb300.so.tmp" in made.names


def test_the_library_without_the_extension(made):
    """Without torch's or Python's headers the library is built, and the error says what is missing."""
    made.fails = "g++"
    for _ in range(2):
        with pytest.raises(RuntimeError, match="lists"):
            b.build_library()
        assert os.path.exists(b.library_path()) and not os.path.exists(b.lists_path())
    assert made.names.count("libmoe_gb300.so.tmp") == 1
    made.fails = None
    b.build_library()
    assert os.path.exists(b.lists_path())


def test_without_torch(made, monkeypatch):
    b.build_library()
    os.remove(b.library_path())

    def none():
        raise ImportError("no torch")

    monkeypatch.setattr(b, "_lists_made_for", none)
    with pytest.raises(ImportError):
        b.build_library()
    assert os.path.exists(b.library_path())
