"""What a build needs: the library nvcc alone, the Python binding PyTorch as well (tiny sources in a folder of their own;
needs nvcc, no GPU)."""
import ctypes
import importlib.util
import os
import shutil
import sysconfig

import pytest

from mbarrier_gemm_pipelines_gb300 import _build

pytestmark = pytest.mark.skipif(not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")),
                                reason="nvcc not available")


@pytest.fixture
def tiny(monkeypatch, tmp_path):
    """A library of one function, built under tmp_path."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text('extern "C" int three() { return 3; }\n')
    (tmp_path / "ext.cpp").write_text("#error not to be compiled\n")
    for name, to in (("CSRC", "csrc"), ("OBJ_DIR", "obj"), ("LIB_PATH", "libtiny.so"), ("EXT_SRC", "ext.cpp"),
                     ("EXT_PATH", "_ext.so")):
        monkeypatch.setattr(_build, name, str(tmp_path / to))
    return tmp_path


def three():
    return ctypes.CDLL(_build.LIB_PATH).three()


def without_torch(monkeypatch, tmp_path):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))


def without_torch_headers(monkeypatch, tmp_path):
    (tmp_path / "torch").mkdir()
    found, spec = importlib.util.find_spec, importlib.util.spec_from_loader("torch", None, is_package=True)
    spec.submodule_search_locations.append(str(tmp_path / "torch"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else found(name, *a))


def without_python_headers(monkeypatch, tmp_path):
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})


@pytest.mark.parametrize("without", [without_torch, without_torch_headers, without_python_headers])
def test_library_without_the_binding(tiny, monkeypatch, without):
    without(monkeypatch, tiny)
    with pytest.warns(UserWarning, match="binding"):
        assert _build.build() == _build.LIB_PATH
    assert three() == 3 and not os.path.exists(_build.EXT_PATH)
    assert _build.up_to_date()


def test_library_is_linked_before_a_binding_that_fails(tiny):
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        _build.build()
    assert three() == 3
    assert not _build.up_to_date()
