"""The build's two parts: the C library, which needs no Python, and the
module over part of it.  A failure of the second leaves the first."""

import ctypes
import glob
import os
import shutil

import pytest

import mla_decode_paged_gb300 as mla

B = mla._build      # the module; mla.build is its function


@pytest.fixture()
def other_build(tmp_path, monkeypatch):
    """A build folder of its own that holds the objects of the package's."""
    mla.build()
    for f in glob.glob(os.path.join(B.BUILD, "*.o")):
        shutil.copy2(f, tmp_path)
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmla_decode.so"))
    return tmp_path


@pytest.mark.parametrize("what,command", [
    ("_ops_compile", ["g++", "-c", "no_such_source.cpp"]),              # binding.cpp does not compile
    ("_ops_compile", ["no_such_compiler_here"]),
    ("_ops_link", ["g++", "-shared", "-lno_such_library_here"]),
])
def test_the_library_is_built_without_the_module(other_build, monkeypatch, what, command):
    for f in glob.glob(str(other_build / "mla_ops*.o")):
        if what == "_ops_compile":
            os.remove(f)
    old = other_build / os.path.basename(B.ops_path())
    old.write_bytes(b"a module of other sources")
    os.utime(old, (1, 1))
    monkeypatch.setattr(B, what, lambda *a: command)
    with pytest.warns(RuntimeWarning, match="library is built, its Python module is not"):
        path = B.build()
    assert path == str(other_build / "libmla_decode.so")
    assert ctypes.CDLL(path).mla_version
    assert not os.path.exists(B.ops_path())


def test_the_module_is_built_beside_the_library(other_build):
    path = B.build()
    assert os.path.dirname(B.ops_path()) == os.path.dirname(path) and os.path.exists(B.ops_path())


def test_the_calls_that_need_the_module_say_so(tmp_path, monkeypatch):
    mla.build()
    mla.library()
    monkeypatch.setattr(mla, "_ops_module", None)
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    with pytest.raises(RuntimeError, match="native module .* is missing"):
        mla.kv_evict(None, None, None, 1)
