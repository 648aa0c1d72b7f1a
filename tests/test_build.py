"""The build on small stand-ins for the sources (no GPU): the library does not hang on
the Python module beside it, and a module built for another torch is not taken."""
import ctypes
import os
import warnings

import pytest
import torch

from paged_kv_cache_213_gb300 import build as b
from paged_kv_cache_213_gb300 import rope

MODULE = '''#include <Python.h>
#include <ATen/core/Tensor.h>
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pagedkv_calls", nullptr, -1, nullptr,
                             nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit__pagedkv_calls() { return PyModule_Create(&module); }
'''


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build.py on a library of one function and a module that does not compile."""
    src, out = tmp_path / "csrc", tmp_path / "_build"
    src.mkdir()
    (src / "one.cpp").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "calls.cpp").write_text("#error no headers here\n")
    for name, value in (("CSRC", src), ("OUT_DIR", out), ("LIB_PATH", out / "libpagedkv.so"),
                        ("CALLS_SRC", tmp_path / "calls.cpp"),
                        ("CALLS_PATH", out / "_pagedkv_calls.so"),
                        ("CALLS_STAMP", out / "_pagedkv_calls.txt")):
        monkeypatch.setattr(b, name, str(value), raising=False)
    return tmp_path


def _library_works():
    return ctypes.CDLL(b.LIB_PATH).one() == 1


def test_the_library_is_built_where_the_module_is_not(tree):
    with pytest.warns(UserWarning, match="Python module"):
        assert b.build() == b.LIB_PATH
    assert _library_works() and not os.path.exists(b.CALLS_PATH)
    assert not b.up_to_date()
    was = os.path.getmtime(b.LIB_PATH)
    with pytest.warns(UserWarning):  # tried again, the library left as it is
        b.build()
    assert os.path.getmtime(b.LIB_PATH) == was


def test_the_library_is_built_without_torch(tree, monkeypatch):
    real = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else real(name, *a))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        b.build()
    assert _library_works() and b.up_to_date()


def test_another_torch_or_python_rebuilds_the_module(tree, monkeypatch):
    (tree / "calls.cpp").write_text(MODULE)
    b.build()
    assert os.path.exists(b.CALLS_PATH) and b.up_to_date()
    assert b.calls_built_for() == b.calls_target() and torch.__version__ in b.calls_target()
    was = os.path.getmtime(b.LIB_PATH)
    target = b.calls_target() + " of another day"
    monkeypatch.setattr(b, "calls_target", lambda: target)
    assert not b.up_to_date()
    b.build()
    assert b.up_to_date() and b.calls_built_for() == target
    assert os.path.getmtime(b.LIB_PATH) == was


@pytest.mark.parametrize("stamp", [None, "torch 1.0, cpython-30", "this one"])
def test_calls_go_through_python_where_the_module_does_not_fit(tree, monkeypatch, stamp):
    """Missing, built for something else, or not loadable: a warning once, and a
    stand-in that takes no call."""
    os.makedirs(b.OUT_DIR)
    if stamp:
        open(b.CALLS_PATH, "w").write("not a module")
        open(b.CALLS_STAMP, "w").write(b.calls_target() if stamp == "this one" else stamp)
    monkeypatch.setattr(rope, "library_path", lambda: b.LIB_PATH)
    monkeypatch.setattr(rope, "library", lambda: None)
    monkeypatch.setattr(rope, "_calls", None)
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        native = rope._native()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert rope._native() is native
    assert native.latent_gather(1, 2, 3) is None and native.qk_append() is None
