"""The library without its compiled Python calls (missing, made for another PyTorch, not buildable): it
builds and loads, and the latent operators' Python forms take the calls (no GPU needed)."""
import os
import sys

import pytest

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build


@pytest.fixture()
def unbound(monkeypatch):
    pskv_build.build()
    monkeypatch.setattr(B, "_calls", None)
    monkeypatch.setattr(B, "_LIB", None)
    return B


def test_the_library_loads_without_them(unbound, monkeypatch):
    monkeypatch.setitem(sys.modules, "paged_split_kv_attn_gb300._calls", None)  # (its import fails)
    monkeypatch.delattr(pskv, "_calls", raising=False)
    assert pskv.load_library().pskv_version() > 0
    with pytest.warns(RuntimeWarning, match="without their compiled calls"):
        calls = B._bind_calls(pskv.load_library())
    assert calls.append(1, 2) is calls.decode() is calls.prefill(3) is calls.verify() is None
    assert B._calls is calls


def test_another_pytorch_s_are_not_imported(unbound, monkeypatch):
    monkeypatch.setattr(pskv_build, "calls_tag", lambda: "cpython-312 somewhere torch 0.0 c++ abi 1")
    assert not pskv_build.calls_fit() and not pskv_build._calls_up_to_date()
    monkeypatch.setitem(sys.modules, "paged_split_kv_attn_gb300._calls", None)
    with pytest.warns(RuntimeWarning, match="another Python or PyTorch"):
        assert B._bind_calls(pskv.load_library()) is B._PythonCalls


def test_they_are_rebuilt_for_another_pytorch(monkeypatch):
    pskv_build.build()
    built = []
    monkeypatch.setattr(pskv_build, "_up_to_date", lambda: True)
    monkeypatch.setattr(pskv_build, "_build_calls", lambda: built.append(1))
    pskv_build.build()
    assert not built  # they fit
    monkeypatch.setattr(pskv_build, "calls_tag", lambda: "cpython-312 somewhere torch 0.0 c++ abi 1")
    pskv_build.build()
    assert built == [1]


def test_the_library_is_built_without_them(monkeypatch):
    pskv_build.build()

    def no_headers():
        raise RuntimeError("no such file: Python.h")

    monkeypatch.setattr(pskv_build, "_up_to_date", lambda: True)
    monkeypatch.setattr(pskv_build, "_calls_up_to_date", lambda: False)
    monkeypatch.setattr(pskv_build, "_build_calls", no_headers)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert os.path.exists(pskv_build.build())


def test_a_library_elsewhere_binds_them_to_itself(unbound):
    """The calls enter the library that was loaded, wherever it lies."""
    calls = B._bind_calls(pskv.load_library())
    assert calls is not B._PythonCalls and calls.decode() is None  # (not a call's arguments)


def test_what_an_earlier_build_left_is_not_used(monkeypatch, tmp_path):
    """Calls that could not be rebuilt beside a new library are not called into it."""
    tag = tmp_path / "_calls.tag"
    tag.write_text(pskv_build.calls_tag())
    pskv_build.build()
    monkeypatch.setattr(pskv_build, "CALLS_TAG", str(tag))
    assert pskv_build.calls_fit()

    def fails():
        raise RuntimeError("no compiler")

    monkeypatch.setattr(pskv_build, "_build_calls", fails)
    with pytest.warns(RuntimeWarning, match="no compiler"):
        pskv_build._try_calls()
    assert not pskv_build.calls_fit()
