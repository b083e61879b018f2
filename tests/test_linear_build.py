"""Building the library where the 8-bit linear layer's torch binding cannot be built (CPU): the compression calls need
only hipcc.  A stand-in for hipcc writes the file that it is asked for."""
import os
import stat

import pytest

import __graft_entry__
from fp8_compression_tensor_taco_amd import build


@pytest.fixture
def no_host_compiler(tmp_path, monkeypatch):
    hipcc = tmp_path / "hipcc"
    hipcc.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\necho library > "$2"\n')
    hipcc.chmod(hipcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("HIPCC", str(hipcc))
    monkeypatch.setenv("CXX", str(tmp_path / "absent"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libtaco.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_linear_binding.so"))
    return tmp_path


def test_library_is_built_without_the_binding(no_host_compiler):
    old = no_host_compiler / "_linear_binding.so"
    old.write_text("of an earlier library")
    with pytest.warns(UserWarning, match="binding"):
        assert build.build_library(verbose=False) == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH)
    assert not old.exists()                          # it may not fit the new library


def test_a_compiler_that_fails_is_no_less_named(no_host_compiler, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    with pytest.warns(UserWarning, match="false failed"):
        build.build_library(verbose=False)


def test_the_whole_build_needs_the_binding(no_host_compiler):
    with pytest.raises((OSError, RuntimeError)):
        __graft_entry__.build()
