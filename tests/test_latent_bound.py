"""Scratch of decode_attn_latent that a serving loop sizes once: a bound over every call of no more
rows, tokens and keys (no GPU needed)."""
import ctypes
import os
import shutil

import pytest

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build
from test_sanitizers import HERE, ROOT, _build_and_run

INVALID, UNSUPPORTED = B.PSKV_ERR_INVALID_ARG, B.PSKV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pskv_build.build()
    return pskv.load_library()


def make(lib, **kw):
    base = dict(num_pages=8, page_size=64, num_kv_heads=1, head_dim_k=576, head_dim_v=512,
                kv_dtype=B.PSKV_DTYPE_BF16, format=B.PSKV_FORMAT_LATENT, k_pool=0x10000, v_pool=None, status=None)
    base.update(kw)
    d = B.LayoutDesc(*[base[f] for f, _ in B.LayoutDesc._fields_])
    h = ctypes.c_void_p()
    assert lib.paged_kv_layout_create(ctypes.byref(d), ctypes.byref(h)) == 0
    return h


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_no_plan_passes_the_bound(tmp_path):
    csrc = os.path.join(ROOT, "paged_split_kv_attn_gb300", "csrc")
    out = _build_and_run(tmp_path, "g++", [os.path.join(HERE, "latent_plan_driver.cpp"),
                                           os.path.join(csrc, "pskv_plan.cpp")],
                         [csrc, os.path.join(ROOT, "include")], "latent_plan_driver", ["-std=c++17"])
    assert "latent plan driver ok" in out


@pytest.mark.parametrize("splits", [1, 2, 4, 5, 1024])
def test_given_splits(lib, splits):
    """With given splits a shorter row can have more pieces too: five tiles in three pieces of two, four in four."""
    h, n = make(lib), ctypes.c_size_t()
    assert lib.decode_attn_latent_workspace_bound(h, 600, 5, 3, 20, splits, ctypes.byref(n)) == 0
    bound = n.value
    assert (bound > 0) == (splits > 1)
    for lens in ([600] * 5, [512] * 5, [511, 3], [300, 200, 1, 0, 600], [129], [1]):
        for tokens in (1, 2, 3):
            arr = (ctypes.c_int32 * len(lens))(*[max(v, tokens) for v in lens])
            assert lib.decode_attn_latent_workspace_bytes(h, arr, 10, len(lens), tokens, 20, splits, ctypes.byref(n)) == 0
            assert n.value <= bound
    lib.paged_kv_layout_destroy(h)


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(max_len=0), INVALID), (dict(batch=0), INVALID), (dict(batch=65536), INVALID),
    (dict(tokens=0), INVALID), (dict(tokens=65), INVALID), (dict(heads=0), INVALID), (dict(heads=129), UNSUPPORTED),
    (dict(splits=-1), INVALID), (dict(splits=1025), INVALID), (dict(batch=65535, tokens=64, heads=128), 0),
])
def test_refusals(lib, kw, code):
    a = dict(max_len=1000, batch=4, tokens=2, heads=16, splits=3)
    a.update(kw)
    h, n = make(lib), ctypes.c_size_t()
    assert lib.decode_attn_latent_workspace_bound(h, a["max_len"], a["batch"], a["tokens"], a["heads"], a["splits"],
                                                  ctypes.byref(n)) == code
    lib.paged_kv_layout_destroy(h)


def test_other_pools_are_refused(lib):
    h, n = make(lib, format=B.PSKV_FORMAT_SPLIT, head_dim_k=512, v_pool=0x20000), ctypes.c_size_t()
    assert lib.decode_attn_latent_workspace_bound(h, 1000, 4, 2, 16, 3, ctypes.byref(n)) == UNSUPPORTED
    lib.paged_kv_layout_destroy(h)
