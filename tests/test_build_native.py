"""When the build makes _native.so anew (no compiler runs: the commands are recorded)."""
import os
import subprocess
import types

import pytest

from top_routing_grouped_02_gb300 import _build


class Tools:
    """Stands in for the compilers: writes what a command would, or fails it."""

    def __init__(self):
        self.commands, self.fail = [], lambda cmd: None

    def __call__(self, cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        self.commands.append((os.path.basename(cmd[0]), os.path.basename(out).split(".tmp")[0]))
        error = self.fail(cmd)
        if isinstance(error, Exception):
            raise error
        if error is None:
            with open(out, "w") as f:
                f.write("built")
        return types.SimpleNamespace(returncode=0 if error is None else 1, stdout="", stderr=error or "")

    def take(self):
        got, self.commands = self.commands, []
        return got


@pytest.fixture
def tools(tmp_path, monkeypatch):
    t = Tools()
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    os.utime(torch / "version.py", (0, 0))
    monkeypatch.setattr(subprocess, "run", t)
    monkeypatch.setattr(_build, "nvcc", lambda: "/cuda/bin/nvcc")
    monkeypatch.setattr(_build, "_torch_dirs", lambda: (str(torch / "include"), str(torch / "lib")))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(_build, "NATIVE", str(tmp_path / "_native.so"))
    t.torch = torch
    return t


def test_another_torch_makes_it_anew(tools):
    _build.build()
    first = tools.take()
    assert ("g++", "binding.o") in first and ("g++", "_native.so") in first and ("nvcc", "libmoe.so") in first
    _build.build()
    assert tools.take() == []
    # another version in the same place, with an old date as an installer may leave it
    (tools.torch / "version.py").write_text("__version__ = '2'\n")
    os.utime(tools.torch / "version.py", (0, 0))
    _build.build()
    assert tools.take() == [("g++", "binding.o"), ("g++", "_native.so")]
    _build.build()
    assert tools.take() == []


@pytest.mark.parametrize("error", [FileNotFoundError("no g++"), "Python.h: No such file or directory"])
@pytest.mark.parametrize("output", ["binding.o", "_native.so"])
def test_the_layer_is_built_without_it(tools, capsys, error, output):
    tools.fail = lambda cmd: error if cmd[0] == "g++" and output in cmd[cmd.index("-o") + 1] else None
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.NATIVE)
    assert "_native.so was not built" in capsys.readouterr().out
    # once the tools are there
    tools.fail = lambda cmd: None
    tools.take()
    _build.build()
    assert ("g++", "_native.so") in tools.take() and os.path.exists(_build.NATIVE)


def test_an_old_one_is_not_left_behind(tools):
    _build.build()
    tools.fail = lambda cmd: "error" if cmd[0] == "g++" else None
    (tools.torch / "version.py").write_text("__version__ = '2'\n")
    _build.build()
    assert not os.path.exists(_build.NATIVE)


def test_failures_of_nvcc_stop_the_build(tools):
    tools.fail = lambda cmd: "error" if cmd[0].endswith("nvcc") else None
    with pytest.raises(RuntimeError, match="nvcc failed"):
        _build.build()


def test_the_loaders_message_is_passed_on(monkeypatch):
    from top_routing_grouped_02_gb300 import moe
    import builtins

    real = builtins.__import__

    def fake(name, globals=None, locals=None, fromlist=(), level=0):
        if "_native" in (fromlist or ()):
            raise ImportError("undefined symbol: of another torch")
        return real(name, globals, locals, fromlist, level)

    monkeypatch.setattr(moe, "_nat", None)
    monkeypatch.setattr(moe, "lib", lambda: None)
    monkeypatch.setattr(builtins, "__import__", fake)
    with pytest.raises(RuntimeError, match="undefined symbol: of another torch"):
        moe._native()
