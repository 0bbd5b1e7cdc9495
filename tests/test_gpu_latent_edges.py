"""Calls of the latent operators at the edges of what their documentation allows."""
import threading

import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import HALF_BF16, ROT, LatentCase, check_attention, normal
from test_gpu_latent import expanded_reference, turned, vmax

pytestmark = pytest.mark.gpu


# ---- the page write ----------------------------------------------------------------

@pytest.mark.parametrize("host", [False, True])
@pytest.mark.parametrize("heads", [1, 5])
def test_one_token_of_an_odd_projection(heads, host):
    """A single token's queries inside a row whose width is no multiple of 16 bytes: there is no next row
    for the stride to reach."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(61)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    wide, wide_out = normal(gen, 1, heads * 192 + 4), normal(gen, 1, heads * 64 + 12)
    q, q_out = wide[:, :heads * 192].view(1, heads, 192)[..., 128:], wide_out[:, :heads * 64].view(1, heads, 64)
    rest = wide_out[:, heads * 64:].clone()
    pool, x, ang = normal(gen, 2, 1, 64, 576), normal(gen, 1, 576), torch.rand(9, 32, generator=gen, device="cuda")
    layout = pskv.paged_kv_layout_create(pool, None)
    pskv.kv_prep_append_latent(layout, x, dev([0]), dev([3]), dev([[0, 1]]), dev([2]), 1e-6, None, ang, ang, q=q,
                               q_out=q_out, host=([0], [3], [2]) if host else None)
    want = turned(q.double(), ang[3:4], ang[3:4], "halves")
    # one rounding to bf16; two products and a sum of values below 8 in f32 before it
    assert ((q_out.double() - want).abs() <= HALF_BF16 * want.abs() + 2.0 ** -19 * 8).all()
    assert torch.equal(wide_out[:, heads * 64:], rest)


def test_rows_that_overlap_are_refused():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(62)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pool, ang = normal(gen, 2, 1, 64, 576), torch.rand(9, 32, generator=gen, device="cuda")
    layout, x, q = pskv.paged_kv_layout_create(pool, None), normal(gen, 2, 576), normal(gen, 2, 3, 64)
    for shape, stride in (((2, 3, 64), (0, 64, 1)), ((2, 3, 64), (192, 32, 1))):
        with pytest.raises(ValueError):
            pskv.kv_prep_append_latent(layout, x, dev([0, 0]), dev([3, 4]), dev([[0, 1]]), dev([2]), 1e-6, None, ang, ang,
                                       q=q, q_out=torch.empty(384, dtype=torch.bfloat16, device="cuda").as_strided(shape, stride))


def test_rows_past_32_bits():
    """A pool of more than 2^31 elements (4.4 GB): rows in its last pages are written and read there."""
    pages, page, dc = 60_000, 64, 512
    pool = torch.zeros(pages, 1, page, dc + ROT, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 2 ** 31
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    layout = pskv.paged_kv_layout_create(pool, None, status)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(63)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    n, heads = 150, 20
    table, lease = dev([[pages - 1, pages - 3, pages - 2], [pages - 4, 0, pages - 5]]), dev([3, 3])
    x, ang = normal(gen, 2 * n, dc + ROT), torch.rand(n, 32, generator=gen, device="cuda")
    dense = torch.empty_like(x)
    pskv.kv_prep_append_latent(layout, x, dev([0] * n + [1] * n), dev(list(range(n)) * 2), table, lease, 1e-6, None, ang,
                               ang, dense=dense)
    c = LatentCase(63, [n, n], dc, page, heads)  # (its reference and its inputs' form)
    for b in range(2):
        k = dense[b * n:(b + 1) * n]
        for s in range(3):
            rows = k[s * page:(s + 1) * page]
            assert torch.equal(pool[int(table[b, s]), 0, :rows.shape[0]], rows)
        c.keys[b] = k
    for splits in (0, 1):
        out = pskv.decode_attn_latent(layout, c.q, table, c.lens, c.lens_host, c.scale, num_splits=splits)
        check_attention(out, c.reference(), vmax(c))
    assert int(status[0]) == 0


# ---- absorbed attention ------------------------------------------------------------

BAD_IDS = [-1, -2 ** 31, 2 ** 31 - 1, None]  # None: the first id past the pool


@pytest.mark.parametrize("page", [16, 32, 48, 64, 96, 256])
@pytest.mark.parametrize("dc,heads,tokens", [(512, 32, 1), (256, 20, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_pages_of_every_width(page, dc, heads, tokens, dtype):
    """Refused pages in a tile's first half, its second, both, and its last partial one."""
    lens = [300, 517, 400, 129, 40, 777]
    c = LatentCase(64 + page, lens, dc, page, heads, tokens)
    hidden = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in lens]

    def refuse(b, key, k):
        slot = key // page
        c.table[b, slot] = c.pool.shape[0] if BAD_IDS[k] is None else BAD_IDS[k]
        hidden[b][slot * page:(slot + 1) * page] = True

    refuse(0, 130, 0)                                          # the second tile's first half
    refuse(1, 128 + 80, 1)                                     # its second half
    refuse(1, 516, 2)                                          # the row's last page
    for k, key in enumerate(range(128, 256, 16)):              # a whole tile
        refuse(2, key, k % 4)
    refuse(3, 0, 3)                                            # the first page
    refuse(3, 128, 0)                                          # a last tile of one key
    refuse(5, 5 * 128 + 70, 1)
    ref = c.reference(hidden)
    for splits in (0, 1, 3):
        out = c.run(num_splits=splits, out_dtype=dtype)
        check_attention(out, ref, vmax(c))
        flags = pskv.pskv_check_flags(c.layout, clear=True)
        alone = any(bool(h[:n - t].all()) for h, n in zip(hidden, lens) for t in range(tokens))
        assert flags == pskv.PSKV_FAULT_BAD_PAGE | (pskv.PSKV_FAULT_EMPTY_ROW if alone else 0)


@pytest.mark.parametrize("scale", [-0.05, 0.0])
@pytest.mark.parametrize("lens,dc,page,heads,tokens", [([900, 64, 0, 129], 512, 64, 32, 1), ([700, 33], 256, 48, 20, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scales_that_are_not_positive(scale, lens, dc, page, heads, tokens, dtype):
    c = LatentCase(65, lens, dc, page, heads, tokens, scale=scale)
    for splits in (0, 1, 4):
        check_attention(c.run(num_splits=splits, out_dtype=dtype), c.reference(), vmax(c))
    assert int(c.status[0]) == 0


# ---- several threads ----------------------------------------------------------------

def test_calls_from_several_threads():
    """Each thread its own stream and outputs, all over the same inputs: the compiled calls let
    others run while they enter the library."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(66)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    c = LatentCase(66, [700, 65, 0], heads=24, tokens=2)
    q, kv, rot = normal(gen, 90, 2, 192), normal(gen, 120, 2, 256), normal(gen, 120, 64)
    cu = dev([0, 30, 90]), dev([0, 50, 120])
    target = torch.softmax(torch.randn(5, 3, 901, generator=gen, device="cuda"), -1)
    drafts, u = torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.rand(5, 3, generator=gen, device="cuda")
    work = [lambda: [c.run()], lambda: [c.run(num_splits=1, out_dtype=torch.float32)],
            lambda: [pskv.prefill_attn_expanded(q, kv, rot, cu[0], [0, 30, 90], cu[1], [0, 50, 120], 0.1)],
            lambda: list(pskv.verify_drafts(target, None, drafts, u))]
    want = [[t.clone() for t in f()] for f in work]
    torch.cuda.synchronize()
    wrong = []

    def run(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for i in range(100):
                    j = (i + k) % len(work)
                    got = work[j]()
                    if i % 10 == 0:
                        stream.synchronize()
                        if not all(torch.equal(a, b) for a, b in zip(want[j], got)):
                            wrong.append((k, i, j))
            stream.synchronize()
        except Exception as e:  # told to the test's thread
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
    assert int(c.status[0]) == 0
