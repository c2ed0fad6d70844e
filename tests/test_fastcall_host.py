"""Which native Python calls are loaded: those built for the running torch and
Python, or none, with a warning; on the CPU."""
import sysconfig
import warnings

import pytest
import torch

from row_reduction_norm_gb300 import api, build as B


@pytest.fixture(autouse=True)
def as_before():
    held = api._fast
    yield
    api._fast = held


def test_the_file_is_for_one_torch_and_one_python(monkeypatch):
    here = B.fastcall_path()
    assert here.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and str(torch.__version__) in here
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert B.fastcall_path() != here


def test_the_module_of_this_torch_is_loaded_and_bound():
    path = B.build_fastcall()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        fast = api._bind_fast()
    assert fast.__file__ == path and api._fast is fast


@pytest.mark.parametrize("there", ["nothing", "something else"])
def test_without_one_the_python_bodies_are_used(monkeypatch, tmp_path, there):
    path = tmp_path / "_fastcall.so"
    if there == "something else":
        path.write_bytes(b"not a module")
    monkeypatch.setattr(B, "fastcall_path", lambda: str(path))
    with pytest.warns(RuntimeWarning, match="native Python calls"):
        fast = api._bind_fast()
    assert api._fast is fast
    for name in ("qk_norm_rope", "qk_norm_rope_backward", "qkv_append", "rms_norm_dropout", "rms_norm_backward",
                 "rms_norm_dropout_backward"):
        assert not api._took(getattr(fast, name)(1, 2, 3), name)


def test_a_module_of_another_torch_is_left_alone(monkeypatch):
    """Found by its name alone: it is not opened to see."""
    B.build_fastcall()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.warns(RuntimeWarning, match="does not exist"):
        assert isinstance(api._bind_fast(), api._PythonCalls)
