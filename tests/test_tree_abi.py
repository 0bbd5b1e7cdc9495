"""Refusals of sampling, drafted trees and forked rows, all decided on the host before any launch (no GPU needed)."""
import ctypes

import pytest

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build

INVALID, UNSUPPORTED = B.PSKV_ERR_INVALID_ARG, B.PSKV_ERR_UNSUPPORTED
P = 0x30000


@pytest.fixture(scope="module")
def lib():
    pskv_build.build()
    return pskv.load_library()


@pytest.fixture()
def make(lib):
    made = []

    def one(**kw):
        base = dict(num_pages=8, page_size=64, num_kv_heads=1, head_dim_k=576, head_dim_v=512,
                    kv_dtype=B.PSKV_DTYPE_BF16, format=B.PSKV_FORMAT_LATENT, k_pool=0x10000, v_pool=None, status=None)
        base.update(kw)
        d, h = B.LayoutDesc(*[base[f] for f, _ in B.LayoutDesc._fields_]), ctypes.c_void_p()
        assert lib.paged_kv_layout_create(ctypes.byref(d), ctypes.byref(h)) == 0
        made.append(h)
        return h

    yield one
    for h in made:
        lib.paged_kv_layout_destroy(h)


def handles(*hs):
    return (ctypes.c_void_p * len(hs))(*[h if h is None else h.value for h in hs]), len(hs)


U, TOKENS = P + 0x80000, P + 0x90000
SAMPLE = dict(logits=P, dtype=0, row=100, requests=2, each=3, vocab=100, filters=None, u=U, tokens=TOKENS, probs=None,
              probs_dtype=0, status=None)


def sample(lib, **kw):
    a = {**SAMPLE, **kw}
    f = None if a["filters"] is None else ctypes.byref(B.SampleDesc(*a["filters"]))
    return lib.sample_tokens(a["logits"], a["dtype"], a["row"], a["requests"], a["each"], a["vocab"], f, a["u"],
                             a["tokens"], a["probs"], a["probs_dtype"], a["status"], None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(dtype=2), dict(dtype=-1), dict(row=99), dict(row=-1), dict(requests=0), dict(each=0),
    dict(vocab=0), dict(vocab=(1 << 22) + 1, row=1 << 23), dict(requests=1 << 13, each=1 << 12), dict(u=None),
    dict(tokens=None), dict(u=None, tokens=None), dict(probs=P + (1 << 20), probs_dtype=5), dict(probs=P),
    dict(probs=P + 2396), dict(probs=P - 1198, probs_dtype=1, row=200), dict(logits=P + 2400, probs=P + 4), dict(logits=P + 2), dict(u=U + 1),
    dict(tokens=TOKENS + 2), dict(probs=P + (1 << 20) + 2), dict(probs=P + (1 << 20) + 1, probs_dtype=1), dict(status=P + 1),
    dict(filters=(P + 2, None, None, None)), dict(filters=(None, P + 1, None, None)),
    dict(filters=(None, None, P + 3, None)), dict(filters=(None, None, None, P + 2)),
    # what is written among what is read
    dict(tokens=U), dict(tokens=U + 20), dict(tokens=U - 20), dict(tokens=P + 2396), dict(probs=U - 2396),
    dict(probs=TOKENS), dict(probs=TOKENS + 20), dict(filters=(TOKENS + 20, None, None, None)),
    dict(filters=(None, TOKENS - 4, None, None)), dict(filters=(None, None, TOKENS, None)),
    dict(filters=(None, None, None, TOKENS + 8)),
    dict(probs=P + (1 << 20), filters=(None, P + (1 << 20) + 2396, None, None))])
def test_sample_refusals(lib, kw):
    assert sample(lib, **kw) == INVALID


def test_walk_refusals(lib):
    # 0 drafts 1 masks 2 sampled (32, 64 and 32 bytes) 5 tokens 6 path 7 kept (32, 32 and 8)
    base = [P, P + 0x100, P + 0x200, 2, 4, P + 0x300, P + 0x400, P + 0x500, None, None]
    for at, bad in [(5, P), (5, P + 28), (6, P + 0x100 + 60), (7, P + 0x200 - 4), (5, P + 0x200), (6, P + 0x300 + 28),
                    (7, P + 0x400), (7, P + 0x300 + 28), (0, None), (1, None), (2, None), (3, 0), (3, (1 << 20) + 1), (4, 0), (4, 65), (5, None), (6, None),
                    (7, None), (0, P + 2), (1, P + 0x104), (2, P + 0x201), (5, P + 0x302), (6, P + 0x402), (7, P + 0x502), (8, P + 2)]:
        args = list(base)
        args[at] = bad
        assert lib.verify_tree(*args) == INVALID, (at, bad)


def test_tree_over_other_pools_and_without_masks(lib, make):
    lens = (ctypes.c_int32 * 1)(100)
    call = lambda h, mask, n=8: lib.decode_attn_latent_tree(h, P, P, 4, lens, P, mask, 1, n, 8, 0.1, 1, P, 1 << 30, P, 1, None, None)
    latent = make()
    assert call(latent, None) == call(latent, P + 4) == call(latent, P, 65) == call(None, P) == INVALID
    split = make(format=B.PSKV_FORMAT_SPLIT, head_dim_k=512, v_pool=0x20000, num_kv_heads=4)
    assert call(split, P) == UNSUPPORTED
    lens[0] = 7  # shorter than its window
    assert call(latent, P) == INVALID


@pytest.mark.parametrize("kw", [dict(num_pages=9), dict(page_size=32), dict(head_dim_k=320, head_dim_v=256),
                                dict(format=B.PSKV_FORMAT_SPLIT, head_dim_k=512, v_pool=0x20000)])
def test_layers_have_one_description(lib, make, kw):
    hs = handles(make(), make(k_pool=0x90000), make(**kw))
    assert lib.kv_keep_tokens(*hs, P, 4, P, P, P, 2, 8, 0x50000, None) == INVALID
    assert lib.kv_fork_rows(*hs, P, P, P, 2, P, 4, P, P, 2, None) == INVALID


@pytest.mark.parametrize("other", [0x100000, 0x100000 + 8 * 64 * 1152 - 16, 0x100000 - 8 * 64 * 1152 + 16])
def test_layers_share_no_memory(lib, make, other):
    hs = handles(make(k_pool=0x100000), make(k_pool=0x400000), make(k_pool=other))
    assert lib.kv_keep_tokens(*hs, P, 4, P + 0x1000, P + 0x2000, P + 0x3000, 2, 8, P + 0x4000, None) == INVALID
    assert lib.kv_fork_rows(*hs, P, P, P, 2, P + 0x100, 4, P + 0x200, P + 0x300, 2, None) == INVALID
    assert lib.kv_fork_rows(*hs, P, P, P, 0, P, 4, P, P, 2, None) == INVALID


def test_keys_and_values_share_no_memory(lib, make):
    split = dict(format=B.PSKV_FORMAT_SPLIT, head_dim_k=512, num_kv_heads=4)  # regions of 0x200000 bytes
    for k, v in [(0x1000000, 0x1000000), (0x1000000, 0x1200000 - 16), (0x1200000 - 16, 0x1000000)]:
        hs = handles(make(k_pool=k, v_pool=v, **split))
        assert lib.kv_fork_rows(*hs, P, P, P, 0, P, 4, P, P, 2, None) == INVALID
    hs = handles(make(k_pool=0x1400000, v_pool=0x1000000, **split), make(k_pool=0x1600000, v_pool=0x1200000, **split))
    assert lib.kv_fork_rows(*hs, P, P, P, 0, P, 4, P, P, 2, None) == 0


def test_layouts_given_wrongly(lib, make):
    h = make()
    huge = make(page_size=1 << 24)  # more vectors a page than 32 bits count
    for hs, code in [((None, 1), INVALID), (handles(h, None), INVALID), (handles(*[h] * 129), INVALID),
                     ((handles(h)[0], 0), INVALID), (handles(huge), UNSUPPORTED)]:
        assert lib.kv_keep_tokens(*hs, P, 4, P, P, P, 2, 8, 0x50000, None) == code
        assert lib.kv_fork_rows(*hs, P, P, P, 2, P, 4, P, P, 2, None) == code


def test_keep_refusals(lib, make):
    #        0 table 1 stride 2 lens 3 path 4 kept 5 batch 6 tokens 7 new lens
    base = [P, 4, P + 0x1000, P + 0x2000, P + 0x3000, 2, 8, P + 0x4000]
    hs = handles(make())
    for at, bad in [(0, None), (1, 0), (2, None), (3, None), (4, None), (5, 0), (5, 65536), (6, 0), (6, 65), (7, None),
                    (0, P + 2), (2, P + 1), (3, P + 1), (4, P + 1), (7, P + 0x4002), (7, P + 0x1004), (7, P + 0x2000 + 60),
                    (7, P + 0x3004), (7, P + 28)]:
        args = list(base)
        args[at] = bad
        assert lib.kv_keep_tokens(*hs, *args, None) == INVALID, (at, bad)


def test_fork_refusals(lib, make):
    #       0 src 1 dst 2 new 3 n 4 table 5 stride 6 lens 7 leases 8 batch
    base = [P, P, P, 2, P + 0x100, 4, P + 0x200, P + 0x300, 2]
    hs = handles(make())
    for at, bad in [(0, None), (1, None), (2, None), (3, -1), (3, 65536), (4, None), (5, 0), (6, None), (7, None), (8, 0),
                    (0, P + 1), (1, P + 1), (2, P + 2), (4, P + 0x102), (6, P + 0x201), (7, P + 0x303),
                    (0, P + 0x200), (1, P + 0x304), (2, P + 0x100 + 28), (4, P + 4), (4, P + 0x200 - 28), (6, P + 0x304)]:
        args = list(base)
        args[at] = bad
        assert lib.kv_fork_rows(*hs, *args, None) == INVALID, (at, bad)
    assert lib.kv_fork_rows(*hs, None, None, None, 0, None, 4, None, None, 2, None) == 0  # no fork
