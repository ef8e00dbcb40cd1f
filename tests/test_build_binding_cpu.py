"""The native binding is optional: the library is built without it, and said so."""
import os
import subprocess

import pytest

from selective_state_space_56_b200 import build as s6build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Every output under tmp_path; compilers are recorded, not run (a command writes its -o file)."""
    ran = []

    def run(cmd, **kw):
        ran.append(os.path.basename(cmd[0]))
        if ran[-1] in fails:
            raise fails[ran[-1]]
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    fails = {}
    monkeypatch.setattr(s6build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(s6build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(s6build, "BINDING_PATH", str(tmp_path / "native.so"))
    monkeypatch.setattr(s6build.subprocess, "run", run)
    return ran, fails


def test_both_are_built(elsewhere):
    ran, _ = elsewhere
    assert s6build.build() == s6build.LIB_PATH
    assert os.path.exists(s6build.LIB_PATH) and os.path.exists(s6build.BINDING_PATH)
    assert ran.count("g++") == 1 and ran.count("nvcc") == len(s6build.sources()) + 1


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), RuntimeError("no headers")], ids=["no_compiler", "no_headers"])
def test_the_library_is_built_without_the_binding(elsewhere, error):
    ran, fails = elsewhere
    fails["g++"] = error
    open(s6build.BINDING_PATH, "w").close()  # made for older sources
    os.utime(s6build.BINDING_PATH, (1, 1))
    with pytest.warns(UserWarning, match="interpreter"):
        assert s6build.build() == s6build.LIB_PATH
    assert os.path.exists(s6build.LIB_PATH) and not os.path.exists(s6build.BINDING_PATH)


def test_a_failing_library_is_an_error(elsewhere):
    _, fails = elsewhere
    fails["nvcc"] = RuntimeError("nvcc")
    with pytest.raises(RuntimeError):
        s6build.build()


def test_another_torch_gets_a_binding_of_its_own(monkeypatch):
    """What is up to date for one torch is not for another, and is not loaded by it."""
    import importlib

    import torch

    from selective_state_space_56_b200 import ops
    mine = s6build.BINDING_PATH
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    try:
        assert importlib.reload(s6build).BINDING_PATH != mine
        assert not os.path.exists(s6build.BINDING_PATH)
        assert ops._load_native(ops.load_library()) is None
    finally:
        monkeypatch.undo()
        assert importlib.reload(s6build).BINDING_PATH == mine
