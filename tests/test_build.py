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


@pytest.fixture
def torch_dir(tmp_path, monkeypatch):
    """A torch installation whose version the test sets."""
    where = tmp_path / "torch"
    where.mkdir()
    spec = types.SimpleNamespace(submodule_search_locations=[str(where)])
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: spec if name == "torch" else None)
    (where / "version.py").write_text("__version__ = '1'\n")
    return where


def test_another_torch_rebuilds_the_module(sandbox, torch_dir):
    def modules():
        return sum("py_calls.cpp" in str(c) for c in sandbox)

    build.build()
    assert modules() == 1
    build.build()
    assert modules() == 1  # up to date
    (torch_dir / "version.py").write_text("__version__ = '2'\n")
    build.build()
    assert modules() == 2
    build.build()
    assert modules() == 2


def test_a_module_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    """Its calls would read tensors by the layout of the torch it was compiled against."""
    build.build()
    calls = tmp_path / "ds_calls.so"
    calls.write_text("")
    (tmp_path / "ds_calls.torch").write_text("__version__ = 'another'\n")
    monkeypatch.setattr(_lib, "_calls", None)
    monkeypatch.setattr(_lib, "LIB_PATH", str(tmp_path / "libdsample.so"))
    _lib._lib or _lib.load(build.LIB)
    with pytest.raises(OSError, match="another torch"):
        _lib.calls()


def test_the_built_module_is_loaded(monkeypatch):
    build.build()
    monkeypatch.setattr(_lib, "_calls", None)
    assert callable(_lib.calls().sample)
