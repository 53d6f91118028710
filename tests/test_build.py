"""The build's parts do not depend on one another: the C library needs hipcc
alone (no compiler is run here)."""
import builtins
import os
import types

import pytest

from few_row_quantized_amd import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's outputs in a folder of their own, hipcc and the host compiler
    as stand-ins that only leave their output files."""
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libqgemv.so"))
    monkeypatch.setattr(b, "MODULE", str(tmp_path / "_qgemv_torch.so"))
    monkeypatch.setattr(b, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(b, "_compile", lambda src, verbose: str(tmp_path / (src + ".o")))
    fails = []

    def run(cmd, **kw):
        bad = any(f in cmd[0] for f in fails)
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=int(bad), stderr="no", stdout="")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setenv("CXX", "g++")
    return tmp_path, fails


def test_both_parts(tree):
    assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.MODULE)


def test_the_library_stands_where_the_module_does_not_compile(tree):
    tree[1].append("g++")
    with pytest.raises(RuntimeError, match="compile failed"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.MODULE)


def test_the_library_alone_without_torch(tree, monkeypatch, capsys):
    open(b.MODULE, "w").close()  # of an earlier build
    real = builtins.__import__

    def no_torch(name, *a, **kw):
        if name == "torch":
            raise ImportError("No module named 'torch'")
        return real(name, *a, **kw)

    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.MODULE) and "torch not found" in capsys.readouterr().out


def test_the_library_alone_without_a_host_compiler(tree, monkeypatch, capsys):
    monkeypatch.setenv("CXX", "no-such-compiler")
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.MODULE) and "no-such-compiler not found" in capsys.readouterr().out
