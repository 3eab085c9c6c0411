"""The build's order and conditions, with the compilers replaced by a recorder."""
import os

import pytest

import free_block_sparse_gb300 as fbs
from free_block_sparse_gb300 import build


@pytest.fixture
def recorded(tmp_path, monkeypatch):
    """Builds into tmp_path; every command is recorded and its output file made."""
    commands = []

    def run(cmd):
        commands.append(cmd)
        if "binding.cpp" in " ".join(cmd) and "-c" in cmd and getattr(run, "fails", False):
            raise RuntimeError("command failed: binding")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "o"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libsparge.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    return run, commands


def test_the_library_builds_without_torch(recorded, monkeypatch):
    """The C library needs nvcc and a C++ compiler alone."""
    run, commands = recorded
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, package=None: None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING) and not any("torch" in " ".join(c) for c in commands)
    assert len([c for c in commands if "-c" in c]) == len(build.CUDA_SOURCES) + len(build.CXX_SOURCES)


def test_a_binding_that_does_not_compile_leaves_the_library(recorded):
    pytest.importorskip("torch")
    run, _ = recorded
    run.fails = True
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_both_are_built_and_only_once(recorded):
    pytest.importorskip("torch")
    _, commands = recorded
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
    n = len(commands)
    assert n == len(build.CUDA_SOURCES) + len(build.CXX_SOURCES) + 3   # the binding's object and two links
    build.build()
    assert len(commands) == n


def test_calls_without_the_binding_say_so(monkeypatch, tmp_path):
    pytest.importorskip("torch")
    if not os.path.exists(fbs.LIB_PATH):
        build.build()
    monkeypatch.setattr(fbs, "_binding_module", None)
    fbs.lib()
    monkeypatch.setattr(fbs, "_PKG", str(tmp_path))
    with pytest.raises(RuntimeError, match="_binding.so is not built"):
        fbs.cache4_store(None, None, None, None)
