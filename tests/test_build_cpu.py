"""The build and the import where the optional CPython module cannot be made or does not fit."""
import os
import sys
import types

import pytest

import sparse_attention_indexer_packed_gb300 as idx
from sparse_attention_indexer_packed_gb300 import _lib, build


@pytest.fixture
def binding(tmp_path, monkeypatch):
    """Paths of a module that is older than its source."""
    so, src = tmp_path / "_binding.so", tmp_path / "idx_binding.c"
    so.write_bytes(b"old")
    src.write_text("")
    os.utime(so, (1, 1))
    monkeypatch.setattr(build, "BINDING", str(so))
    return so, src


def no_run(cmd):
    raise AssertionError(f"nothing is to be run: {cmd}")


def test_a_machine_without_gcc_builds_without_the_module(binding, monkeypatch, capsys):
    so, src = binding
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build._build_binding([str(src)], ".tmp", no_run, False)
    assert not so.exists()                  # nor is an outdated one left
    assert "gcc not found" in capsys.readouterr().err
    assert not build._build_binding([str(src)], ".tmp", no_run, True)


def test_a_machine_without_python_headers_builds_without_the_module(binding, monkeypatch, capsys, tmp_path):
    so, src = binding
    monkeypatch.setattr(build.shutil, "which", lambda name: "/usr/bin/" + name)
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build._build_binding([str(src)], ".tmp", no_run, False)
    assert not so.exists()
    assert "Python.h not found" in capsys.readouterr().err


def test_a_failing_compiler_is_named(binding, monkeypatch):
    monkeypatch.setattr(build.subprocess, "run",
                        lambda *a, **k: types.SimpleNamespace(returncode=1, stdout="", stderr="no space"))
    monkeypatch.setattr(build, "_nvcc", lambda: "/x/bin/nvcc")
    with pytest.raises(RuntimeError, match="^nvcc failed"):
        build.build_library(force=True)
    monkeypatch.setattr(build, "SOURCES", ["idx_kv.cu"])
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    monkeypatch.setattr(build.shutil, "which", lambda name: "/usr/bin/" + name)
    monkeypatch.setattr(build.os.path, "exists", lambda path: True)
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **k: types.SimpleNamespace(
        returncode=int(cmd[0] == "gcc"), stdout="", stderr=""))
    with pytest.raises(RuntimeError, match="^gcc failed"):
        build.build_library(force=True)


@pytest.mark.parametrize("module", [
    types.SimpleNamespace(),                                             # no bind
    types.SimpleNamespace(bind=lambda dtypes: None),                     # another bind
    types.SimpleNamespace(bind=lambda *a: None),                         # a call is missing
])
def test_a_module_that_does_not_fit_is_passed_over(monkeypatch, module):
    monkeypatch.setattr(idx, "_binding", module, raising=False)
    monkeypatch.setitem(sys.modules, "sparse_attention_indexer_packed_gb300._binding", module)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(_lib, "LIB_PATH", __file__)
    assert _lib._native_calls() == tuple(getattr(_lib, name) for name in _lib.NATIVE_CALLS)


def test_a_build_in_a_process_with_the_old_module_goes_on_through_ctypes(monkeypatch):
    for name in _lib.NATIVE_CALLS:
        monkeypatch.setattr(idx, name, lambda *a: None)
    build._drop_native_calls()
    for name in _lib.NATIVE_CALLS:
        assert getattr(idx, name) is getattr(_lib, name)


def test_warnings_of_the_compilers_are_shown(monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(build, "SOURCES", ["idx_kv.cu"])
    monkeypatch.setattr(build, "_nvcc", lambda: "/x/bin/nvcc")
    monkeypatch.setattr(build, "_drop_native_calls", lambda: None)
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    monkeypatch.setattr(build, "_stale", lambda out, deps: False)
    monkeypatch.setattr(build, "_build_binding", lambda *a: False)
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **k: types.SimpleNamespace(
        returncode=0, stdout="", stderr="ptxas warning : Registers are spilled\n" if "-c" in cmd else ""))
    build.build_library(force=True)
    assert capsys.readouterr().err == "ptxas warning : Registers are spilled\n"
