"""The build of the Python extension beside the library: made again for another
Python or torch, and left out where it cannot be compiled."""
import os
import shutil
import sysconfig

import pytest
import torch

from bit_quantized_mixture_b200 import build as B


@pytest.fixture
def built(monkeypatch, tmp_path):
    """A tree in which everything is up to date; the commands that a build runs are
    collected, their targets made empty."""
    B.build()
    for name in ("LIB", "BINDING"):
        copy = tmp_path / os.path.basename(getattr(B, name))
        shutil.copy2(getattr(B, name), copy)
        monkeypatch.setattr(B, name, str(copy))
    monkeypatch.setattr(B, "STAMP", str(tmp_path / "binding.stamp"))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return type("R", (), dict(returncode=0, stdout="", stderr=""))

    monkeypatch.setattr(B.subprocess, "run", run)
    B.build()                              # writes the stamp of this tree
    ran.clear()
    return ran


def test_nothing_to_do(built):
    B.build()
    assert not built


@pytest.mark.parametrize("what", ["python", "torch"])
def test_another_python_or_torch(built, monkeypatch, what):
    if what == "python":
        monkeypatch.setattr(B.sys, "version", "3.99.0 (another one)")
    else:
        monkeypatch.setattr(torch, "__version__", "99.0.0")
    B.build()
    assert [os.path.basename(c[0]) for c in built] == ["g++"]
    built.clear()
    B.build()
    assert not built


@pytest.mark.parametrize("what", ["g++", "Python.h", "option"])
def test_the_library_needs_neither_compiler_nor_headers_of_the_extension(built, monkeypatch, capsys, what):
    os.remove(B.BINDING)
    if what == "g++":
        which = shutil.which
        monkeypatch.setattr(B.shutil, "which", lambda name: None if name == "g++" else which(name))
    elif what == "Python.h":
        paths = sysconfig.get_paths()
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {**paths, "include": "/nowhere"})
    assert B.build(binding=what != "option") == B.LIB
    assert not built and not os.path.exists(B.BINDING)
    assert ("_binding.so is not built" in capsys.readouterr().err) == (what != "option")
