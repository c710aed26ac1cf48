"""The build without what the native binding of the token-sequence calls needs: libgspn.so comes from nvcc alone."""
import ctypes
import os
import shutil

import pytest

import linear_spatial_propagation_gspn_b200 as g

b = g._build_mod


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one function, built somewhere else."""
    if not shutil.which(os.environ.get("NVCC", "nvcc")):
        pytest.skip("no nvcc")
    (tmp_path / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "sources", lambda: [str(tmp_path / "one.cu")])
    return tmp_path


@pytest.mark.parametrize("compiler", ["no-such-compiler", "false"])
def test_the_library_needs_nvcc_alone(small, monkeypatch, compiler):
    monkeypatch.setenv("CXX", compiler)
    (small / "_binding.so").write_text("one of an older library")
    with pytest.warns(RuntimeWarning, match="_binding.so was not built"):
        b.build(force=True)
    assert ctypes.CDLL(b.LIB).one() == 1
    assert sorted(os.listdir(small)) == ["_build", "libone.so", "one.cu"]
    before = os.stat(b.LIB)
    with pytest.warns(RuntimeWarning):                              # tried again; the library itself is up to date
        b.build()
    assert os.stat(b.LIB) == before


def test_a_library_that_does_not_compile_is_an_error(small, monkeypatch):
    script = small / "cxx"                                          # one that leaves its output behind and goes on
    script.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done; : > "$2"; exec sleep 60\n')
    script.chmod(0o755)
    monkeypatch.setenv("CXX", str(script))
    (small / "one.cu").write_text("int one( {\n")
    with pytest.raises(RuntimeError, match="one.cu"):
        b.build(force=True)
    assert not any(f.endswith(".so") or ".tmp" in f for f in os.listdir(small))


def test_calls_without_the_binding_take_the_checked_path(monkeypatch):
    """With no such module, every native call declines."""
    import sys

    monkeypatch.setitem(sys.modules, "linear_spatial_propagation_gspn_b200._seq_fast", None)
    monkeypatch.delattr(g, "_seq_fast", raising=False)
    fast = g._seq._Fast()
    assert fast.conv_step(None) is None and fast.norm_backward() is None
