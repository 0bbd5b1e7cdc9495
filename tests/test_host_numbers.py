"""Host lengths, offsets and counts that do not fit 32 bits are refused, not cut to their low ones
(no GPU needed)."""
import ctypes
import types

import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build

FAR = [2 ** 31, 2 ** 32 + 100, -2 ** 31 - 1, 2 ** 63 - 1]


@pytest.fixture(scope="module")
def lib():
    pskv_build.build()
    return pskv.load_library()


@pytest.fixture()
def latent(lib):
    d = B.LayoutDesc(8, 64, 1, 576, 512, B.PSKV_DTYPE_BF16, B.PSKV_FORMAT_LATENT, 0x10000, None, None)
    h = ctypes.c_void_p()
    assert lib.paged_kv_layout_create(ctypes.byref(d), ctypes.byref(h)) == 0
    yield types.SimpleNamespace(handle=h, page_size=64)
    lib.paged_kv_layout_destroy(h)


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("form", [list, tuple, lambda v: np.array(v, np.int64), lambda v: torch.tensor(v, dtype=torch.int64)])
@pytest.mark.parametrize("take", [B._host_i32, B._lens_i32])
def test_arrays(take, form, far):
    with pytest.raises(ValueError):
        take(form([5, far]), "seq_lens_host")
    assert list(take(form([5, -2 ** 31, 2 ** 31 - 1]), "seq_lens_host")) == [5, -2 ** 31, 2 ** 31 - 1]
    assert list(take(form([]), "seq_lens_host")) == []


def test_arrays_of_mixed_numbers():
    assert list(B._lens_i32([np.int32(7), 8], "seq_lens_host")) == [7, 8]
    with pytest.raises(ValueError):
        B._lens_i32([np.int64(2 ** 40), 8], "seq_lens_host")


@pytest.mark.parametrize("far", FAR)
def test_sizing(latent, far):
    size = pskv.decode_attn_latent_workspace_bytes
    assert size(latent, [250, 7], 4, 2, 3, 2) > 0
    for bad in (([far, 7], 4, 2, 3, 2), ([250, 7], far, 2, 3, 2), ([250, 7], 4, far, 3, 2), ([250, 7], 4, 2, far, 2),
                ([250, 7], 4, 2, 3, far)):
        with pytest.raises(ValueError):
            size(latent, *bad)


@pytest.mark.parametrize("far", FAR)
def test_options(far):
    with pytest.raises(ValueError):
        B._opts(merge_group=far)
