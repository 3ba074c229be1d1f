"""The build of the library and of its extension module, without a GPU."""
import os
import sysconfig

import pytest

from fp8_quantized_paged_concat_gb300 import _build


def test_the_library_needs_no_extension_module(monkeypatch, tmp_path):
    """Without g++ or PyTorch's headers libkvq.so is linked all the same, with
    a warning that says what the calls of the extension module miss."""
    _build.build()

    def no_compiler(force=False):
        raise RuntimeError("g++ failed on kvq_binding.cpp: no such compiler")

    monkeypatch.setattr(_build, "build_native", no_compiler)
    library = str(tmp_path / "libkvq.so")
    with pytest.warns(UserWarning, match="no such compiler"):
        assert _build.build(library=library) == library
    assert os.path.getsize(library) > 0


def test_the_build_check_fails_without_the_extension_module(monkeypatch):
    import __graft_entry__ as graft

    def no_compiler(force=False):
        raise RuntimeError("no such compiler")

    monkeypatch.setattr(_build, "build_native", no_compiler)
    with pytest.raises(RuntimeError, match="no such compiler"), pytest.warns(UserWarning):
        graft.build()


def test_the_extension_module_is_that_of_this_python_and_pytorch(monkeypatch):
    """Its file names both, so that another interpreter or PyTorch, with
    another ABI, says that it is missing and does not load it."""
    import torch

    import fp8_quantized_paged_concat_gb300 as kvq

    _build.build()
    path = _build.native_path()
    assert os.path.exists(path) and path.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and torch.__version__ in path
    assert kvq._load_native().__file__ == path
    monkeypatch.setattr(kvq, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="is missing: build it"):
        kvq._load_native()
