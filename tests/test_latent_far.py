"""Page tables whose last positions pass 32 bits with the tile they lie in (no GPU needed: decided
before any launch)."""
import ctypes

import pytest

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build


@pytest.mark.parametrize("page,keys,refused", [
    (16, 2 ** 31 - 16, True), (64, 2 ** 31 - 64, True), (16, 2 ** 31 - 112, True), (128, 2 ** 31 - 128, True),
    (16, 2 ** 31 - 144, False), (256, 2 ** 31 - 256, False)])
def test_the_last_tile_ends_within_32_bits(page, keys, refused):
    pskv_build.build()
    lib = pskv.load_library()
    d = B.LayoutDesc(8, page, 1, 576, 512, B.PSKV_DTYPE_BF16, B.PSKV_FORMAT_LATENT, 0x10000, None, None)
    h, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.paged_kv_layout_create(ctypes.byref(d), ctypes.byref(h)) == 0
    lens = (ctypes.c_int32 * 1)(100)
    rc = lib.decode_attn_latent_workspace_bytes(h, lens, keys // page, 1, 1, 8, 4, ctypes.byref(n))
    assert rc == (B.PSKV_ERR_INVALID_ARG if refused else 0)
    lib.paged_kv_layout_destroy(h)
