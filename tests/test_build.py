"""The build keeps the CUDA library and the Python extension apart: one that cannot be compiled does not take the other along."""
import os
import shutil

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from gated_deltanet_linear_15_gb300 import build as b


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A build folder of this test's own, with a CUDA library that is up to date."""
    lib = b.build()
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libgdn.so"))
    monkeypatch.setattr(b, "PY_LIB", str(tmp_path / os.path.basename(b.PY_LIB)))
    monkeypatch.setattr(_lib, "_py", None)
    shutil.copy(lib, b.LIB)
    return tmp_path


def _no_extension():
    with pytest.warns(RuntimeWarning, match="extension"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.PY_LIB)
    with pytest.raises(ImportError, match="missing"):
        _lib.load_py()


def test_library_stands_without_the_extension(built, monkeypatch):
    """A source that does not compile; an extension of an older source does not stay."""
    broken = built / "broken.cpp"
    broken.write_text("#error no headers here\n")
    monkeypatch.setattr(b, "PY_SOURCE", str(broken))
    with open(b.PY_LIB, "w") as f:
        f.write("old")
    os.utime(b.PY_LIB, (1, 1))
    _no_extension()


def test_library_stands_without_a_host_compiler(built, monkeypatch):
    monkeypatch.setenv("PATH", str(built))
    monkeypatch.setattr(b, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    _no_extension()


def test_extension_is_of_one_torch():
    """Another torch finds no extension of this one's, and builds its own."""
    assert torch.__version__ in os.path.basename(b.PY_LIB)
