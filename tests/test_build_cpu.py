"""The build's two libraries do not depend on each other."""
import ctypes
import os
import shutil

import pytest

from gemm_epilogue_transformer_tma_gb300 import build as B

SRC = 'extern "C" int answer() { return 42; }\n'


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small source into tmp_path."""
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("nvcc not found")
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text(SRC)
    (tmp_path / "marshal.cpp").write_text("int unused;\n")
    monkeypatch.setattr(B, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(B, "OBJ", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(B, "MARSHAL_SRC", str(tmp_path / "marshal.cpp"))
    return tmp_path


def test_a_marshalling_module_that_fails_leaves_the_library(elsewhere):
    """A source the host compiler refuses: the error is raised, and the
    library, which needs nothing of it, is there and loads."""
    (elsewhere / "marshal.cpp").write_text("#error no headers\n")
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        B.build()
    assert ctypes.CDLL(B.LIB).answer() == 42
    assert not os.path.exists(B.MARSHAL) and not B.up_to_date()


def test_a_library_that_fails_leaves_the_module(elsewhere):
    (elsewhere / "csrc" / "one.cu").write_text("#error no kernels\n")
    with pytest.raises(RuntimeError, match="one.cu"):
        B.build()
    assert os.path.exists(B.MARSHAL) and not os.path.exists(B.LIB)


def test_only_what_is_older_than_its_sources_is_made(elsewhere):
    B.build()
    assert B.up_to_date()
    lib, mod = os.path.getmtime(B.LIB), os.path.getmtime(B.MARSHAL)
    os.utime(elsewhere / "marshal.cpp", (mod + 10, mod + 10))
    assert not B.up_to_date()
    B.build()
    assert os.path.getmtime(B.LIB) == lib and os.path.getmtime(B.MARSHAL) >= mod
