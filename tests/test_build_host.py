"""The build: the library does not depend on torch, and a torch binding that does not
compile neither stops the library nor leaves an older binding in place."""
import ctypes
import sys
import warnings

import pytest

from tma_pipelined_tensor_tn_gb300 import _build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build of one small source, into a directory of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n__global__ void k() {}\n')
    monkeypatch.setattr(_build, "_sources", lambda: [str(src)])
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(_build, "OPS", str(tmp_path / "_torch_ops.so"))
    return tmp_path


def test_library_builds_without_torch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)       # import torch raises ImportError
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        path = _build.build()
    assert ctypes.CDLL(path).one() == 1
    assert not (small / "_torch_ops.so").exists()


@pytest.mark.parametrize("compiler", ["false", "no-such-compiler"])
def test_library_builds_where_the_binding_does_not(small, monkeypatch, compiler):
    pytest.importorskip("torch")
    for name in ("_torch_ops.so", "_torch_ops.so.stamp"):
        (small / name).write_text("of an older build")
    monkeypatch.setenv("CXX", compiler)
    with pytest.warns(RuntimeWarning, match="torch binding"):
        path = _build.build()
    assert ctypes.CDLL(path).one() == 1
    assert not (small / "_torch_ops.so").exists()
