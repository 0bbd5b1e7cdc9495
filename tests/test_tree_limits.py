"""The header states the sizes that sampling, trees and rows are refused beyond, and what a fork's lease may be (no GPU needed)."""
import ctypes
import os
import re

import pytest

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build

HEADER = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pskv.h")).read()
P = 0x1000000000


def about(name):
    """The comment before a function's declaration."""
    at = HEADER.index(f"\nint {name}(")
    return " ".join(HEADER[HEADER.rindex("/*", 0, at):at].replace("\n *", " ").split())


@pytest.fixture(scope="module")
def lib():
    pskv_build.build()
    return pskv.load_library()


@pytest.mark.parametrize("name,calls", [
    ("PSKV_MAX_VOCAB", ["sample_tokens"]), ("PSKV_MAX_SAMPLED", ["sample_tokens"]), ("PSKV_MAX_TREES", ["verify_tree"]),
    ("PSKV_MAX_KEPT_ROWS", ["kv_keep_tokens"]), ("PSKV_MAX_FORKS", ["kv_fork_rows"]),
    ("PSKV_MAX_LAYOUTS", ["kv_keep_tokens"]), ("PSKV_MAX_WINDOW_TOKENS", ["verify_tree", "kv_keep_tokens"])])
def test_limits_are_stated(name, calls):
    assert int(re.search(rf"#define {name} (\d+)", HEADER)[1]) == getattr(B, name)
    assert all(name in about(c) for c in calls)


def test_sizes_past_the_limits_are_refused(lib):
    sample = lambda requests, each, vocab: lib.sample_tokens(P, 0, vocab, requests, each, vocab, None, P << 8, P << 9, None, 0, None, None)
    assert sample(1, 1, B.PSKV_MAX_VOCAB + 1) == B.PSKV_ERR_INVALID_ARG
    assert sample(B.PSKV_MAX_SAMPLED + 1, 1, 1) == sample(1, B.PSKV_MAX_SAMPLED + 1, 1) == B.PSKV_ERR_INVALID_ARG
    assert sample(B.PSKV_MAX_SAMPLED // 64 + 1, 64, 1) == B.PSKV_ERR_INVALID_ARG
    assert lib.verify_tree(P, 2 * P, 3 * P, B.PSKV_MAX_TREES + 1, 1, 4 * P, 5 * P, 6 * P, None, None) == B.PSKV_ERR_INVALID_ARG
    d = B.LayoutDesc(8, 64, 1, 576, 512, B.PSKV_DTYPE_BF16, B.PSKV_FORMAT_LATENT, 0x10000, None, None)
    h = ctypes.c_void_p()
    assert lib.paged_kv_layout_create(ctypes.byref(d), ctypes.byref(h)) == 0
    one = (ctypes.c_void_p * 1)(h.value)
    assert lib.kv_keep_tokens(one, 1, P, 4, 2 * P, 3 * P, 4 * P, B.PSKV_MAX_KEPT_ROWS + 1, 1, 5 * P, None) == B.PSKV_ERR_INVALID_ARG
    assert lib.kv_fork_rows(one, 1, P, 2 * P, 3 * P, B.PSKV_MAX_FORKS + 1, 4 * P, 4, 5 * P, 6 * P, 1 << 20, None) == B.PSKV_ERR_INVALID_ARG
    lib.paged_kv_layout_destroy(h)


def test_refused_lengths_and_leases_are_stated():
    assert "table_stride * page_size at most; else PSKV_FAULT_BAD_LENGTH" in about("kv_keep_tokens")
    assert "or of more than table_stride (PSKV_FAULT_PAST_PAGES)" in about("kv_fork_rows")
