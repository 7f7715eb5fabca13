"""What a build leaves where one of its parts fails (a stand-in for the compiler, which writes its
output and fails where it is told to)."""

import os

import pytest

from causal_conv1d_verify_amd import build as b


@pytest.fixture
def parts(tmp_path, monkeypatch):
    hipcc = tmp_path / "hipcc"
    hipcc.write_text('#!/bin/sh\ncase "$*" in *"$FAIL_AT"*) echo told to fail >&2; exit 1;; esac\n'
                     'while [ "$1" != -o ]; do shift; done\necho made > "$2"\n')
    hipcc.chmod(0o755)
    monkeypatch.setattr(b, "HIPCC", str(hipcc))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    libs = {}
    for name in ("LIB", "LIB_WC", "LIB_LA", "LIB_CALL"):
        libs[name] = str(tmp_path / (name + ".so"))
        monkeypatch.setattr(b, name, libs[name])
    monkeypatch.setenv("FAIL_AT", "no such part")
    return libs


def _there(parts):
    return [name for name, path in parts.items() if os.path.exists(path)]


def test_a_whole_build(parts):
    b.build(verbose=False)
    assert _there(parts) == ["LIB", "LIB_WC", "LIB_LA", "LIB_CALL"]


@pytest.mark.parametrize("at", ["la_call.cpp", "la_call.o -L", "headers"])
def test_the_libraries_are_there_without_the_call_module(parts, at, monkeypatch):
    """Its compilation, its link, or Python's and torch's headers for it: the libraries are built, the
    error is raised, and no older module is left beside them."""
    monkeypatch.setenv("FAIL_AT", at)
    if at == "headers":
        def absent():
            raise ImportError("no torch")

        monkeypatch.setattr(b, "_call_module", absent)
    open(parts["LIB_CALL"], "w").write("an older one")
    with pytest.raises((RuntimeError, ImportError)):
        b.build(verbose=False)
    assert _there(parts) == ["LIB", "LIB_WC", "LIB_LA"]


def test_a_library_that_fails_is_an_error(parts, monkeypatch):
    monkeypatch.setenv("FAIL_AT", "la_few.hip")
    with pytest.raises(RuntimeError, match="told to fail"):
        b.build(verbose=False)
