"""The library needs neither torch's headers nor Python's: where the list helper of the binding does
not compile, libnaju.so is there all the same, and the failure is reported."""
import ctypes
import os

import pytest

from selective_state_space_naju_amd import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one source, away from the tree's own files."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not found")
    monkeypatch.setattr(build, "SOURCES", ["naju_step.hip"])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libnaju.so"))
    monkeypatch.setattr(build, "TENSORS", str(tmp_path / "_tensors.so"))
    compiled = str(tmp_path / "x.o")
    source = str(tmp_path / "x.c")
    with open(source, "w") as f:
        f.write("int naju_here(void) { return 7; }\n")
    os.system("gcc -fPIC -c %s -o %s" % (source, compiled))
    monkeypatch.setattr(build, "_compile", lambda src, verbose: compiled)
    return tmp_path


def test_a_helper_that_does_not_compile_leaves_the_library(small, monkeypatch):
    def broken():
        raise RuntimeError("g++ failed for naju_tensors.cpp")
    monkeypatch.setattr(build, "_compile_tensors", broken)
    with pytest.raises(RuntimeError, match="naju_tensors"):
        build.build()
    assert ctypes.CDLL(build.LIB).naju_here() == 7


def test_the_helper_is_built_too(small, monkeypatch):
    done = []
    monkeypatch.setattr(build, "_compile_tensors", lambda: done.append(1))
    assert build.build() == build.LIB and done == [1]
    assert ctypes.CDLL(build.LIB).naju_here() == 7
