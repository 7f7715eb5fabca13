"""What a build leaves of libseqops.so and its call module where one of its parts fails (a stand-in for the
compiler, which writes its output and fails where it is told to)."""

import os

import pytest

from causal_conv1d_verify_amd import build as b


@pytest.fixture
def made(tmp_path, monkeypatch):
    hipcc = tmp_path / "hipcc"
    hipcc.write_text('#!/bin/sh\ncase "$*" in *"$FAIL_AT"*) echo told to fail >&2; exit 1;; esac\n'
                     'while [ "$1" != -o ]; do shift; done\necho made > "$2"\n')
    hipcc.chmod(0o755)
    monkeypatch.setattr(b, "HIPCC", str(hipcc))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    for name in ("LIB", "LIB_WC", "LIB_LA", "LIB_CALL"):
        monkeypatch.setattr(b, name, str(tmp_path / (name + ".so")))
    monkeypatch.setenv("FAIL_AT", "no such part")
    return lambda: sorted(f for f in os.listdir(tmp_path) if f.endswith(".so"))


LIBS = ["LIB.so", "LIB_LA.so", "LIB_WC.so", "libseqops.so"]


def test_a_whole_build(made):
    b.build(verbose=False)
    assert made() == sorted([*LIBS, "LIB_CALL.so", "_sqcall.so"])


@pytest.mark.parametrize("at,left", [("sq_call.cpp", "LIB_CALL.so"), ("sq_call.o -L", "LIB_CALL.so"), ("la_call.cpp", "_sqcall.so")])
def test_one_call_module_does_without_the_other(made, at, left, monkeypatch, tmp_path):
    monkeypatch.setenv("FAIL_AT", at)
    for name in ("LIB_CALL.so", "_sqcall.so"):
        (tmp_path / name).write_text("an older one")
    with pytest.raises(RuntimeError, match="told to fail"):
        b.build(verbose=False)
    assert made() == sorted([*LIBS, left])


def test_a_kernel_that_fails_is_an_error(made, monkeypatch):
    monkeypatch.setenv("FAIL_AT", "sq_prompt.hip")
    with pytest.raises(RuntimeError, match="told to fail"):
        b.build(verbose=False)
