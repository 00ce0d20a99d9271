"""CPU: the C library is built by nvcc alone; the extension that marshals the
torch forms' calls is optional, at build time and at run time."""
import os
import sys
import sysconfig
import warnings

import pytest

import mixed_precision_matmul_gb300 as mpg
from mixed_precision_matmul_gb300 import _build, fp8


@pytest.fixture
def fresh_lib(tmp_path, monkeypatch):
    """build() has to link again, into a folder of its own."""
    mpg.build()
    target = tmp_path / "libmpgemm.so"
    monkeypatch.setattr(_build, "LIB", str(target))
    return target


def fail(error):
    def f():
        raise error
    return f


@pytest.mark.parametrize("error", [RuntimeError("g++ failed for torch_calls.cpp"), FileNotFoundError("g++")])
def test_library_is_linked_where_the_extension_does_not_compile(fresh_lib, monkeypatch, error):
    monkeypatch.setattr(_build, "build_torch_calls", fail(error))
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        assert _build.build() == str(fresh_lib)
    assert fresh_lib.stat().st_size > 1 << 20


def test_library_is_linked_without_torch(fresh_lib, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)           # import torch: ModuleNotFoundError
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _build.build()
    assert fresh_lib.exists()


def test_calls_without_the_extension_take_the_python_form(tmp_path, monkeypatch):
    import torch
    mpg.build()
    monkeypatch.setattr(_build, "torch_calls_path", lambda: str(tmp_path / "_torch_calls-other.so"))
    fp8._calls.cache_clear()
    try:
        with pytest.warns(RuntimeWarning, match="marshalled in Python"):
            with pytest.raises(ValueError, match="2-D"):       # the Python form's own words
                mpg.fp8_quantize(torch.zeros(4))
        a, s = torch.zeros((4, 256), dtype=torch.float8_e4m3fn), torch.zeros((4, 2))
        with pytest.raises(ValueError, match="CUDA"):
            mpg.gemm_fp8(a, s, a, s)
    finally:
        fp8._calls.cache_clear()


def test_the_extension_is_named_for_its_python():
    assert os.path.basename(_build.torch_calls_path()).endswith(sysconfig.get_config_var("EXT_SUFFIX"))
