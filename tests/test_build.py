"""What a build makes, and when (nothing is compiled: the compilers are recorded)."""
import os
import subprocess
import sys
import types

import pytest

from dual_ar_tts_gb300 import build as b


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The commands that builds into an empty folder run, by their compiler; `fail` names one that fails."""
    commands, state = [], types.SimpleNamespace(fail=None)

    def run(cmd, **_):
        name = os.path.basename(cmd[0])
        commands.append(name)
        if name == state.fail:
            return subprocess.CompletedProcess(cmd, 1, "", "no")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name in ("OUT", "CALLS", "BUILD"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    state.commands = commands
    return state


def _count(made):
    n = made.commands.count("nvcc"), made.commands.count("g++")
    made.commands.clear()
    return n


ALL = len(b.SOURCES) + 1        # and the link


def test_library_without_torch(made, monkeypatch):
    """The library needs no torch and no Python headers."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert os.path.exists(b.build()) and _count(made) == (ALL, 0)
    assert not os.path.exists(b.CALLS)
    b.build()
    assert _count(made) == (0, 0)


def test_library_without_python_headers(made, monkeypatch, tmp_path):
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    b.build()
    assert _count(made) == (ALL, 0)


def test_calls_follow_torch(made, monkeypatch):
    """The calls are made again for another torch or Python, or after they failed; the library is not."""
    pytest.importorskip("torch")
    if b._torch() is None:
        pytest.skip("no Python.h")
    b.build()
    assert _count(made) == (ALL, 2) and os.path.exists(b.CALLS)
    b.build()
    assert _count(made) == (0, 0)
    was = b._against
    monkeypatch.setattr(b, "_against", lambda torch: was(torch) + "another")
    b.build()
    assert _count(made) == (0, 2)
    b.build()
    assert _count(made) == (0, 0)
    os.remove(b.CALLS)
    b.build()
    assert _count(made) == (0, 2)


def test_failing_calls_leave_the_library(made):
    pytest.importorskip("torch")
    if b._torch() is None:
        pytest.skip("no Python.h")
    made.fail = "g++"
    with pytest.raises(RuntimeError):
        b.build()
    assert os.path.exists(b.OUT) and not os.path.exists(b.CALLS)
    made.fail = None
    made.commands.clear()
    b.build()
    assert _count(made) == (0, 2)
