"""The build beside a machine's Python: the C library without torch, and the module of torch calls against the torch that
is installed. Compilers are stand-ins that write the file they were asked for."""
import importlib.util
import os
import subprocess
import types

import pytest

from vocab_wide_logit_gb300 import _lib, build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """A build into an empty folder; the commands that it ran."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1] if "-o" in cmd else cmd[-1]
        with open(out, "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(build, "OUT", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libdsample.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "ds_calls.so"))
    return ran


def test_without_torch_the_c_library_is_built(sandbox, monkeypatch):
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    lib = build.build()
    assert os.path.exists(lib) and not os.path.exists(build.CALLS)
    assert not any("py_calls.cpp" in str(c) for c in sandbox)


def test_a_failing_module_leaves_the_c_library(sandbox, monkeypatch):
    good = subprocess.run

    def run(cmd, **kw):
        r = good(cmd, **kw)
        if any("py_calls.cpp" in c for c in cmd):
            r.returncode = 1
        return r

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises(RuntimeError):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)
