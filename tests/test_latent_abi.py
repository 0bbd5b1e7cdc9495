"""Refusals and sizes of the latent-cache entry points and verify_drafts, all
decided on the host before any launch (no GPU needed)."""
import ctypes

import pytest

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build

INVALID, UNSUPPORTED = B.PSKV_ERR_INVALID_ARG, B.PSKV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pskv_build.build()
    return pskv.load_library()


def make(lib, **kw):
    base = dict(num_pages=8, page_size=64, num_kv_heads=1, head_dim_k=576, head_dim_v=512,
                kv_dtype=B.PSKV_DTYPE_BF16, format=B.PSKV_FORMAT_LATENT, k_pool=0x10000, v_pool=None,
                status=None)
    base.update(kw)
    d = B.LayoutDesc(*[base[f] for f, _ in B.LayoutDesc._fields_])
    h = ctypes.c_void_p()
    return lib.paged_kv_layout_create(ctypes.byref(d), ctypes.byref(h)), h


@pytest.fixture()
def latent(lib):
    rc, h = make(lib)
    assert rc == 0
    yield h
    lib.paged_kv_layout_destroy(h)


def i32s(*v):
    return (ctypes.c_int32 * len(v))(*v)


@pytest.mark.parametrize("kw,code", [
    (dict(), 0),
    (dict(head_dim_k=320, head_dim_v=256), 0),
    (dict(page_size=16), 0),
    (dict(v_pool=0x20000), INVALID),                 # the values lie in the rows
    (dict(k_pool=None), INVALID),
    (dict(k_pool=0x10008), INVALID),
    (dict(page_size=40), INVALID),
    (dict(head_dim_k=512), UNSUPPORTED),
    (dict(head_dim_k=640), UNSUPPORTED),
    (dict(head_dim_k=192, head_dim_v=128), UNSUPPORTED),
    (dict(num_kv_heads=2), UNSUPPORTED),
    (dict(kv_dtype=B.PSKV_DTYPE_F32), UNSUPPORTED),
    (dict(format=B.PSKV_FORMAT_SPLIT), INVALID),     # a split pool without its V region
])
def test_latent_layouts(lib, kw, code):
    rc, h = make(lib, **kw)
    assert rc == code
    if rc == 0:
        lib.paged_kv_layout_destroy(h)


def test_other_calls_refuse_a_latent_pool(lib, latent):
    lens, p = i32s(100), 0x30000
    assert lib.decode_attn_splitkv(latent, p, p, 4, lens, p, 1, 8, 0.1, 1, p, 1 << 30, p, 1, None,
                                   None) == UNSUPPORTED
    assert lib.decode_attn_multirow(latent, p, p, 4, lens, p, 1, 2, 8, 0.1, 1, p, 1 << 30, p, 1, None,
                                    None) == UNSUPPORTED
    assert lib.prefill_attn_paged(latent, p, i32s(0, 5), p, p, 4, lens, p, 1, 8, 0, 0.1, 1, p, 1 << 30,
                                  p, 1, None, None) == UNSUPPORTED
    assert lib.kv_append_rows(latent, p, p, p, p, 1, p, 4, p, 1, None, None, None, None) == UNSUPPORTED
    prep = B.PrepDesc(0, 1e-6, None, None, None, None, 0)
    assert lib.kv_prep_append(latent, ctypes.byref(prep), p, 4096, 0, 0, 0, 1, 1, p, p, None, p, 4, p, 1,
                              None, None, None, p, None) == UNSUPPORTED
    n = ctypes.c_int32()
    assert lib.pskv_plan_splits(latent, 1, 8, lens, ctypes.byref(n)) == UNSUPPORTED


def test_latent_calls_refuse_other_pools(lib):
    rc, h = make(lib, format=B.PSKV_FORMAT_SPLIT, head_dim_k=512, v_pool=0x20000)
    assert rc == 0
    lens, p = i32s(100), 0x30000
    assert lib.decode_attn_latent(h, p, p, 4, lens, p, 1, 1, 8, 0.1, 1, p, 1 << 30, p, 1, None,
                                  None) == UNSUPPORTED
    prep = B.LatentPrepDesc(1e-6, 0, None, p, p, 10, 0)
    assert lib.kv_prep_append_latent(h, ctypes.byref(prep), p, 576, 1, p, p, None, p, 4, p, 1, None,
                                     None, None, None, None) == UNSUPPORTED
    lib.paged_kv_layout_destroy(h)


def decode_rc(lib, h, lens, **kw):
    a = dict(q=0x30000, tables=0x40000, stride=4, dev=0x50000, batch=len(lens), tokens=1, hq=32, scale=0.1,
             splits=4, ws=0x60000, ws_bytes=1 << 30, out=0x70000, dtype=1)
    a.update(kw)
    return lib.decode_attn_latent(h, a["q"], a["tables"], a["stride"], i32s(*lens), a["dev"], a["batch"],
                                  a["tokens"], a["hq"], a["scale"], a["splits"], a["ws"], a["ws_bytes"],
                                  a["out"], a["dtype"], None, None)


@pytest.mark.parametrize("lens,kw,code", [
    ([100], dict(q=None), INVALID), ([100], dict(tables=None), INVALID), ([100], dict(dev=None), INVALID),
    ([100], dict(out=None), INVALID), ([100], dict(q=0x30008), INVALID), ([100], dict(out=0x70004), INVALID),
    ([257], {}, INVALID),                    # past the table
    ([-1], {}, INVALID),
    ([4], dict(tokens=5), INVALID),          # fewer keys than tokens
    ([100], dict(tokens=0), INVALID), ([100], dict(tokens=65), INVALID),
    ([100], dict(hq=0), INVALID), ([100], dict(hq=129), UNSUPPORTED),
    ([100], dict(scale=float("nan")), INVALID), ([100], dict(splits=-1), INVALID),
    ([100], dict(splits=1025), INVALID), ([100], dict(dtype=7), INVALID),
    ([200], dict(ws=None), B.PSKV_ERR_WORKSPACE_TOO_SMALL),
    ([200], dict(ws_bytes=1000), B.PSKV_ERR_WORKSPACE_TOO_SMALL),
    ([100], dict(stride=1 << 26), INVALID),  # positions past 32 bits
    ([100], dict(batch=0), INVALID),
])
def test_decode_refusals(lib, latent, lens, kw, code):
    assert decode_rc(lib, latent, lens, **kw) == code


def test_decode_refuses_an_appending_option(lib, latent):
    p = 0x30000
    opts = B.DecodeOpts(0, None, None, p, p, p)
    assert lib.decode_attn_latent(latent, p, p, 4, i32s(100), p, 1, 1, 8, 0.1, 1, p, 1 << 30, p, 1,
                                  ctypes.byref(opts), None) == UNSUPPORTED


def test_workspace_bytes(lib, latent):
    n = ctypes.c_size_t()
    get = lambda splits, lens=(250, 0), tokens=2, hq=3: (lib.decode_attn_latent_workspace_bytes(
        latent, i32s(*lens), 4, len(lens), tokens, hq, splits, ctypes.byref(n)), n.value)
    assert get(1) == (0, 0)
    rc, size = get(4)
    partial = pskv.pskv_partial_scratch_bytes(2, 32, 512, 2)[3]  # 2 x 3 columns in a group of 32; 250 keys: two tiles
    assert rc == 0 and partial <= size <= partial + 4 * 256
    assert get(4, lens=(1,), tokens=2)[0] == INVALID


def prep_rc(lib, h, prep=None, **kw):
    p = 0x30000
    f = dict(eps=1e-6, pairs=0, w=p, rope_cos=p, rope_sin=p, max_pos=10, num_q_heads=4, q=p, q_token=256,
             q_head=64, q_out=p, q_out_token=256, q_out_head=64)
    f.update(prep or {})
    a = dict(x=p, x_token=576, n=2, row_of=p, pos_of=p, tables=p, stride=4, pages=p, batch=2, hosts=(None,) * 3,
             dense=None)
    a.update(kw)
    d = B.LatentPrepDesc(*[f[k] for k, _ in B.LatentPrepDesc._fields_])
    return lib.kv_prep_append_latent(h, ctypes.byref(d), a["x"], a["x_token"], a["n"], a["row_of"],
                                     a["pos_of"], None, a["tables"], a["stride"], a["pages"], a["batch"],
                                     *a["hosts"], a["dense"], None)


@pytest.mark.parametrize("prep,kw,code", [
    ({}, dict(n=0), 0), ({}, dict(n=-1), INVALID), ({}, dict(x=None), INVALID), ({}, dict(x=0x30008), INVALID),
    ({}, dict(x_token=568), INVALID), ({}, dict(x_token=580), INVALID), ({}, dict(dense=0x30002), INVALID),
    (dict(eps=-1.0), {}, INVALID), (dict(eps=float("nan")), {}, INVALID), (dict(pairs=2), {}, INVALID),
    (dict(rope_cos=None), {}, INVALID), (dict(max_pos=0), {}, INVALID), (dict(num_q_heads=-1), {}, INVALID),
    (dict(q=None), {}, INVALID), (dict(q_out=None), {}, INVALID), (dict(q=0x30004), {}, INVALID),
    (dict(q_head=60), {}, INVALID), (dict(q_out_token=12), {}, INVALID), (dict(w=0x30004), {}, INVALID),
    ({}, dict(row_of=None), INVALID), ({}, dict(pages=None), INVALID), ({}, dict(batch=0), INVALID),
    ({}, dict(hosts=(i32s(0, 1), None, None)), INVALID),
    ({}, dict(hosts=(i32s(0, 2), i32s(0, 0), i32s(1, 1))), INVALID),          # no such row
    ({}, dict(hosts=(i32s(0, 1), i32s(0, 64), i32s(1, 1))), B.PSKV_ERR_PAST_PAGES),
])
def test_prep_refusals(lib, latent, prep, kw, code):
    assert prep_rc(lib, latent, prep, **kw) == code


def expanded_rc(lib, cq, ck, **kw):
    a = dict(q=0x30000, kv=0x30000, rot=0x30000, rot_token=64, dq=0x30000, dk=0x30000, heads=4, scale=0.1,
             out=0x30000, dtype=1, status=None, batch=len(cq) - 1)
    a.update(kw)
    return lib.prefill_attn_expanded(a["q"], a["kv"], a["rot"], a["rot_token"], i32s(*cq), a["dq"], i32s(*ck),
                                     a["dk"], a["batch"], a["heads"], a["scale"], a["out"], a["dtype"],
                                     a["status"], None)


@pytest.mark.parametrize("cq,ck,kw,code", [
    ([0, 0], [0, 5], {}, 0),                 # no query: nothing to do
    ([0, 5], [0, 4], {}, INVALID),           # fewer keys than queries
    ([1, 5], [0, 9], {}, INVALID), ([0, 5], [1, 9], {}, INVALID), ([0, 5, 4], [0, 5, 9], {}, INVALID),
    ([0, 5], [0, 5], dict(q=None), INVALID), ([0, 5], [0, 5], dict(kv=0x30008), INVALID),
    ([0, 5], [0, 5], dict(rot_token=60), INVALID), ([0, 5], [0, 5], dict(rot_token=68), INVALID),
    ([0, 5], [0, 5], dict(dq=None), INVALID), ([0, 5], [0, 5], dict(heads=0), INVALID),
    ([0, 5], [0, 5], dict(scale=float("inf")), INVALID), ([0, 5], [0, 5], dict(dtype=3), INVALID),
    ([0, 5], [0, 5], dict(status=0x30002), INVALID), ([0, 5], [0, 5], dict(batch=0), INVALID),
])
def test_expanded_refusals(lib, cq, ck, kw, code):
    assert expanded_rc(lib, cq, ck, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(target=None), dict(u=None), dict(tokens=None), dict(accepted=None), dict(drafts=None), dict(dtype=2),
    dict(batch=0), dict(max_drafts=-1), dict(max_drafts=65), dict(vocab=0), dict(target=0x30002),
    dict(draft=0x30001), dict(u=0x30002), dict(num=0x30001), dict(batch=(1 << 20) + 1), dict(vocab=(1 << 30) + 1),
])
def test_verify_refusals(lib, kw):
    p = 0x30000
    a = dict(target=p, draft=p, dtype=0, drafts=p, num=None, u=p, batch=2, max_drafts=3, vocab=10, tokens=p,
             accepted=p, status=None)
    a.update(kw)
    assert lib.verify_drafts(a["target"], a["draft"], a["dtype"], a["drafts"], a["num"], a["u"], a["batch"],
                             a["max_drafts"], a["vocab"], a["tokens"], a["accepted"], a["status"],
                             None) == INVALID
