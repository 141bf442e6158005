"""The compiled part of the binding is built where it can be, anew for another torch, and the package goes on
without it.  No GPU."""
import os
import subprocess

import pytest

from cluster_routed_sparse_b200 import build, streaming


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build whose _fast.so and stamp are in tmp_path; calls of the compiler are listed, not made."""
    calls = []

    def run(cmd, check):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "FAST", str(tmp_path / "_fast.so"))
    monkeypatch.setattr(build, "STAMP", str(tmp_path / "_build" / "fast"))
    monkeypatch.setattr(subprocess, "run", run)
    return calls


def test_built_once_and_again_for_another_torch(elsewhere, monkeypatch):
    import torch
    build._build_fast()
    assert len(elsewhere) == 1 and os.path.exists(build.FAST)
    build._build_fast()
    assert len(elsewhere) == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    build._build_fast()
    assert len(elsewhere) == 2
    build._build_fast()
    assert len(elsewhere) == 2
    build._build_fast(force=True)
    assert len(elsewhere) == 3


def test_without_headers_or_a_compiler_the_package_goes_on(elsewhere, monkeypatch, capfd):
    build._build_fast()
    for error in (subprocess.CalledProcessError(1, "g++"), FileNotFoundError("g++")):
        def run(cmd, check, error=error):
            raise error
        monkeypatch.setattr(subprocess, "run", run)
        build._build_fast(force=True)
        assert not os.path.exists(build.FAST)  # none that was built for something else
        assert "ctypes" in capfd.readouterr().err


def test_one_that_does_not_load_is_named(monkeypatch, tmp_path):
    def none(*_):
        raise ImportError("undefined symbol")
    monkeypatch.setattr(streaming.importlib, "import_module", none)
    monkeypatch.setattr(streaming, "FAST", str(tmp_path / "_fast.so"))
    assert streaming._load_fast() is None  # not built: nothing to say
    open(streaming.FAST, "w").close()
    with pytest.warns(RuntimeWarning, match="does not load"):
        assert streaming._load_fast() is None


def test_without_torch_the_library_is_built(elsewhere, monkeypatch, capfd):
    import sys
    for calls in (0, 1):  # nothing built before, and something
        with monkeypatch.context() as m:
            m.setitem(sys.modules, "torch", None)  # importing it fails
            build._build_fast()
        assert len(elsewhere) == calls and "ctypes" in capfd.readouterr().err
        build._build_fast()
