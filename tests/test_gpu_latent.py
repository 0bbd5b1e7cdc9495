"""The latent cache on the GPU: page write, absorbed attention, expanded
attention, against f64 references (tests/latent_cases.py)."""
import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import HALF_BF16, ROT, LatentCase, check_attention, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return pskv.load_library()


def vmax(case):
    return max([float(k.abs().max()) for k in case.keys if k.numel()] or [0.0])


# ---- absorbed attention -----------------------------------------------------------

@pytest.mark.parametrize("lens,dc,page,heads,tokens,splits", [
    ([1], 512, 64, 32, 1, 1),                      # one key
    ([63, 64, 65], 512, 64, 32, 1, 1),             # around a tile
    ([127, 129, 1, 0], 512, 256, 32, 1, 0),        # a padded row
    ([300, 17], 256, 16, 16, 1, 0),                # pages of one key group
    ([333, 500], 512, 48, 8, 1, 3),                # pages that end inside a tile
    ([200], 512, 64, 1, 1, 0),                     # one head
    ([1000], 512, 256, 3, 5, 0),                   # odd heads x odd tokens
    ([700, 90], 512, 64, 128, 1, 0),
    ([260, 3], 512, 64, 128, 3, 2),                # three blocks of columns
    ([64, 200], 512, 64, 20, 64, 0),               # the longest window, one row all window
    ([5000], 256, 64, 100, 2, 0),
    ([40], 512, 64, 32, 1, 7),                     # more partitions than tiles
    ([2049, 2000, 5, 0, 900], 512, 256, 32, 4, 0),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_matches_f64(lens, dc, page, heads, tokens, splits, dtype):
    c = LatentCase(len(lens) + heads, lens, dc, page, heads, tokens)
    out = c.run(num_splits=splits, out_dtype=dtype)
    check_attention(out, c.reference(), vmax(c))
    assert int(c.status[0]) == 0
    again = c.run(num_splits=splits, out_dtype=dtype)
    assert torch.equal(out, again)
    for b, n in enumerate(lens):
        if n == 0:
            assert not out[b].any()


def test_one_key_gives_its_latent():
    c = LatentCase(3, [1, 1], heads=40)
    out = c.run()
    for b in range(2):
        assert torch.equal(out[b, 0], c.keys[b][0, :512].expand(40, 512))


def test_long_row_and_its_splits():
    c = LatentCase(5, [40002], page=256, heads=32)
    ref = c.reference()
    for splits in (0, 1, 2, 76, 200):
        check_attention(c.run(num_splits=splits), ref, vmax(c))


@pytest.mark.parametrize("heads", [32, 128])
def test_peaked_and_growing_scores(heads):
    """Scores that grow along the row by far more than any slack, and one key that outweighs all."""
    c = LatentCase(6, [900], heads=heads, scale=1.0)
    for b, k in enumerate(c.keys):
        ramp = torch.linspace(0.01, 0.5, k.shape[0], device="cuda")[:, None]
        new = (k.float() * ramp).to(torch.bfloat16)
        new[700] = (c.q[0, 0, 0].float() * 0.5).to(torch.bfloat16)
        k.copy_(new)
        i = torch.arange(k.shape[0], device="cuda")
        c.pool.view(-1, 576)[c.table[b].long()[i // 64] * 64 + i % 64] = new
    # |q.k| reaches about 576 * 0.5 here: 640 * 2^-24 * 576 = 2.2e-2 of a score at worst
    out, ref = c.run(out_dtype=torch.float32), c.reference()
    assert (out.double() - ref).abs().max() <= 2 * (2.2e-2 + 2.0 ** -16) * vmax(c)
    assert float((out.double() - ref).norm() / ref.norm()) <= 1e-3


def test_bad_pages_are_skipped_and_flagged():
    c = LatentCase(7, [300, 200])
    c.table[0, 2] = -5
    c.table[1, 0] = c.pool.shape[0]
    hidden = [torch.zeros(300, dtype=torch.bool, device="cuda"), torch.zeros(200, dtype=torch.bool, device="cuda")]
    hidden[0][128:192] = True
    hidden[1][:64] = True
    check_attention(c.run(), c.reference(hidden), vmax(c))
    assert pskv.pskv_check_flags(c.layout, clear=True) == pskv.PSKV_FAULT_BAD_PAGE


def test_a_row_of_bad_pages_gives_zeros():
    c = LatentCase(8, [100, 70])
    c.table[0, :] = -1
    for splits in (1, 2):
        out = c.run(num_splits=splits)
        assert not out[0].any()
        assert pskv.pskv_check_flags(c.layout, clear=True) & pskv.PSKV_FAULT_BAD_PAGE


def test_device_lengths_out_of_range_are_clamped_and_flagged():
    c = LatentCase(9, [100, 130], tokens=3)
    for bad in (-7, 10 ** 6, 2):
        lens = torch.tensor([bad, 130], dtype=torch.int32, device="cuda")
        out = pskv.decode_attn_latent(c.layout, c.q, c.table, lens, c.lens_host, c.scale)
        check_attention(out[1:], c.reference()[1:], vmax(c))
        assert pskv.pskv_check_flags(c.layout, clear=True) & pskv.PSKV_FAULT_BAD_LENGTH


def test_shorter_and_longer_device_lengths_replay_one_plan():
    """A captured call follows the device lengths; its partition count stays the plan's."""
    c = LatentCase(10, [900, 64, 700])
    ws = pskv.latent_workspace(c.layout, c.lens_host, 1, 32, table_stride=c.table.shape[1])
    out = torch.empty(3, 1, 32, 512, dtype=torch.bfloat16, device="cuda")
    c.run(workspace=ws, out=out)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.run(workspace=ws, out=out)
    for lens in ([900, 64, 700], [1, 64, 699], [640, 0, 65], [900, 1, 700]):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        full, c.keys, c.lens_host = (c.keys, c.lens_host), [k[:n] for k, n in zip(c.keys, lens)], lens
        ref = c.reference()
        c.keys, c.lens_host = full
        out.fill_(float("nan"))
        graph.replay()
        check_attention(out, ref, vmax(c))
    assert int(c.status[0]) == 0


@pytest.mark.parametrize("splits", [0, 1, 3])
def test_many_rows(splits):
    """More rows than a warp's lanes, two blocks of columns, rows of one piece between rows of several."""
    c = LatentCase(13, [2 + 37 * b % 700 if b % 9 else 0 for b in range(45)], dc=256, page=32, heads=70, tokens=2)
    out = c.run(num_splits=splits)
    check_attention(out, c.reference(), vmax(c))
    assert int(c.status[0]) == 0 and torch.equal(out, c.run(num_splits=splits))


def test_bad_pages_between_pieces():
    c = LatentCase(14, [3000, 1500], page=64)
    c.table[0, 20:30] = c.pool.shape[0] + 3       # whole pieces of them
    c.table[1, 7] = -2 ** 31
    hidden = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in (3000, 1500)]
    hidden[0][1280:1920] = True
    hidden[1][448:512] = True
    for splits in (0, 1, 24):
        check_attention(c.run(num_splits=splits), c.reference(hidden), vmax(c))
        assert pskv.pskv_check_flags(c.layout, clear=True) == pskv.PSKV_FAULT_BAD_PAGE


def test_two_graphs_share_a_workspace():
    """Captured calls of different shapes, replayed in turn on one stream over one scratch tensor."""
    cases = [LatentCase(15, [900, 2000]), LatentCase(16, [3000], heads=50, tokens=3)]
    size = max(pskv.latent_workspace(c.layout, c.lens_host, c.tokens, c.heads, table_stride=c.table.shape[1]).numel()
               for c in cases)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    side, graphs, outs = torch.cuda.Stream(), [], []
    for c in cases:
        out = c.run(workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.run(workspace=ws, out=out)
        graphs.append(graph)
        outs.append(out)
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            out.fill_(float("nan"))
            graph.replay()
    for c, out in zip(cases, outs):
        check_attention(out, c.reference(), vmax(c))


def test_workspace_and_output_guards():
    """Nothing outside the workspace's bytes or the output is written."""
    c = LatentCase(11, [700, 300], heads=24, tokens=2)
    n = pskv.decode_attn_latent_workspace_bytes(c.layout, c.lens_host, c.table.shape[1], 2, 24)
    assert n > 0
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    big = torch.full((4, 2, 24, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    pool = c.pool.clone()
    c.run(workspace=ws[:n], out=big[1:3])
    check_attention(big[1:3], c.reference(), vmax(c))
    assert (ws[n:] == 0x5A).all() and (big[0] == 7).all() and (big[3] == 7).all()
    assert torch.equal(pool.view(torch.int16), c.pool.view(torch.int16))


def test_streams():
    c = LatentCase(12, [3000, 50])
    ref = c.reference()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = c.run(stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        b = c.run()
    side.synchronize()
    check_attention(a, ref, vmax(c))
    assert torch.equal(a, b)


def test_python_refusals():
    c = LatentCase(13, [100])
    with pytest.raises(ValueError):
        pskv.decode_attn_latent(c.layout, c.q[..., :512].contiguous(), c.table, c.lens, [100], 0.1)
    with pytest.raises(ValueError):
        c.run(out=torch.empty(1, 1, 32, 576, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        pskv.decode_attn_latent(c.layout, c.q, c.table, c.lens, [100, 3], 0.1)
    with pytest.raises(TypeError):
        pskv.decode_attn_latent(c.layout, c.q.float(), c.table, c.lens, [100], 0.1)
    with pytest.raises(TypeError):
        pskv.decode_attn_latent(c.layout, c.q, c.table.cpu(), c.lens, [100], 0.1)
    with pytest.raises(pskv.PskvError):
        pskv.decode_attn_splitkv(c.layout, c.q[:, 0], c.table, c.lens, [100], 0.1)


# ---- the page write ----------------------------------------------------------------

def turned(y, cos, sin, pairs):
    """f64 rotation; cos, sin [n, 32] spread over y [n, (heads,) 64]."""
    cos, sin = [t.double().reshape(t.shape[0], *[1] * (y.dim() - 2), 32) for t in (cos, sin)]
    i = torch.arange(32, device="cuda")
    first, second = (i, i + 32) if pairs == "halves" else (2 * i, 2 * i + 1)
    out = torch.empty_like(y)
    out[..., first] = y[..., first] * cos - y[..., second] * sin
    out[..., second] = y[..., second] * cos + y[..., first] * sin
    return out


@pytest.mark.parametrize("n,dc,page,heads,pairs,dense,norm", [
    (1, 512, 64, 1, "halves", False, True), (7, 512, 256, 32, "adjacent", True, True),
    (130, 256, 16, 3, "halves", True, False), (33, 512, 48, 0, "adjacent", False, True),
    (501, 256, 64, 13, "adjacent", True, True), (64, 512, 256, 128, "halves", False, True)])
def test_prep_append(n, dc, page, heads, pairs, dense, norm):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    rows, first = 3, torch.tensor([0, 40, 7], dtype=torch.int32, device="cuda")
    pages = -(-(n + 5) // page)
    pool = normal(gen, 3 * pages + 2, 1, page, dc + ROT)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    layout = pskv.paged_kv_layout_create(pool, None, status)
    table = torch.randperm(3 * pages + 2, generator=torch.Generator().manual_seed(n))[:3 * pages].reshape(3, pages)
    table = table.to(torch.int32).cuda()
    lease = torch.full((3,), pages, dtype=torch.int32, device="cuda")
    wide = normal(gen, n, dc + ROT + 24, scale=3.0)                  # rows strided
    x = wide[:, 8:8 + dc + ROT]
    row_of = (torch.arange(n, device="cuda") % rows).to(torch.int32)
    pos_of = (torch.arange(n, device="cuda") // rows + 2).to(torch.int32)
    w = torch.randn(dc, generator=gen, device="cuda") if norm else None
    angle = torch.arange(n + 60, device="cuda").double()[:, None] * 1e4 ** (-torch.arange(32, device="cuda").double() / 32)
    cos, sin = angle.cos().float(), angle.sin().float()
    q_rows = normal(gen, n, max(heads, 1), 192)
    q_out = normal(gen, n, max(heads, 1), dc + ROT)
    keep, q_keep, x_keep = pool.clone(), q_out.clone(), wide.clone()
    den = torch.empty(n, dc + ROT, dtype=torch.bfloat16, device="cuda") if dense else None
    pskv.kv_prep_append_latent(layout, x, row_of, pos_of, table, lease, 1e-5, w, cos, sin, pairs=pairs,
                               first_pos=first, q=q_rows[:, :heads, 128:] if heads else None,
                               q_out=q_out[:, :heads, dc:] if heads else None, dense=den,
                               host=(row_of.cpu(), pos_of.cpu(), lease.cpu()))
    assert int(status[0]) == 0
    p = (pos_of + first[row_of.long()]).long()
    xd = x.double()
    want = torch.cat([xd[:, :dc] / torch.sqrt((xd[:, :dc] ** 2).mean(1, keepdim=True) + 1e-5) * (1 if w is None else w.double()),
                      turned(xd[:, dc:], cos[p], sin[p], pairs)], 1)
    where = table[row_of.long(), pos_of.long() // page].long() * page + pos_of.long() % page
    got = pool.view(-1, dc + ROT)[where]
    # one rounding to bf16, and some f32 roundings of values up to |a| + |b| before it
    assert ((got.double() - want).abs() <= HALF_BF16 * want.abs() + 2.0 ** -19 * (1 + xd.abs().amax())).all()
    other = torch.ones(pool.view(-1, dc + ROT).shape[0], dtype=torch.bool, device="cuda")
    other[where] = False
    assert torch.equal(pool.view(-1, dc + ROT)[other], keep.view(-1, dc + ROT)[other])
    assert torch.equal(wide, x_keep)
    if dense:
        assert torch.equal(den, got)
    if heads:
        wq = turned(q_rows[:, :heads, 128:].double(), cos[p], sin[p], pairs)
        assert ((q_out[:, :heads, dc:].double() - wq).abs() <= HALF_BF16 * wq.abs() + 2.0 ** -19 * 8).all()
        assert torch.equal(q_out[..., :dc], q_keep[..., :dc])
        same = q_rows.clone()                                        # in place, as the expanded form wants it
        pskv.kv_prep_append_latent(layout, x, row_of, pos_of, table, lease, 1e-5, w, cos, sin, pairs=pairs,
                                   first_pos=first, q=same[:, :heads, 128:], q_out=same[:, :heads, 128:])
        assert torch.equal(same[:, :heads, 128:], q_out[:, :heads, dc:])
        assert torch.equal(same[..., :128], q_rows[..., :128])


def test_prep_refused_rows_write_nothing():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    pool = normal(gen, 4, 1, 64, 576)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    layout = pskv.paged_kv_layout_create(pool, None, status)
    table = torch.tensor([[0, 1], [9, 2]], dtype=torch.int32, device="cuda")
    lease = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    ang = torch.zeros(100, 32, device="cuda")
    bad = [((0, 64), pskv.PSKV_FAULT_PAST_PAGES), ((1, 3), pskv.PSKV_FAULT_BAD_PAGE),
           ((2, 0), pskv.PSKV_FAULT_PAST_PAGES), ((-1, 0), pskv.PSKV_FAULT_PAST_PAGES),
           ((0, -1), pskv.PSKV_FAULT_PAST_PAGES), ((1, 127), pskv.PSKV_FAULT_BAD_POSITION)]
    for (row, pos), bit in bad:
        x, q = normal(gen, 1, 576), normal(gen, 1, 4, 64)
        keep, out, dense = pool.clone(), torch.zeros_like(q), torch.zeros_like(x)
        pskv.kv_prep_append_latent(layout, x, torch.tensor([row], dtype=torch.int32, device="cuda"),
                                   torch.tensor([pos], dtype=torch.int32, device="cuda"), table, lease, 1e-6,
                                   None, ang, ang, q=q, q_out=out, dense=dense)
        assert pskv.pskv_check_flags(layout, clear=True) == bit
        assert torch.equal(pool, keep) and not out.any() and not dense.any()


# ---- expanded attention --------------------------------------------------------------

def expanded_reference(q, kv, k_rot, cq, ck, scale):
    out = torch.zeros(q.shape[0], q.shape[1], 128, dtype=torch.float64, device="cuda")
    for a, e, c, f in zip(cq, cq[1:], ck, ck[1:]):
        if e == a:
            continue
        own = (f - c) - (e - a) + torch.arange(e - a, device="cuda")
        hide = torch.arange(f - c, device="cuda") > own[:, None]
        for h in range(q.shape[1]):
            k = torch.cat([kv[c:f, h, :128], k_rot[c:f]], 1).double()
            s = (q[a:e, h].double() @ k.T) * scale
            out[a:e, h] = torch.softmax(s.masked_fill(hide, -float("inf")), -1) @ kv[c:f, h, 128:].double()
    return out


@pytest.mark.parametrize("new,old,heads", [
    ([1], [0], 1), ([1, 1, 1], [0, 62, 63], 3), ([64], [0], 4), ([127, 128, 129], [1, 0, 300], 2),
    ([0, 5, 0, 200], [10, 0, 0, 77], 5), ([256], [256], 8), ([257, 255, 1], [0, 513, 2000], 3), ([1000], [17], 2),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_expanded_matches_f64(new, old, heads, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sum(new))
    cq = [0] + np.cumsum(new).tolist()
    ck = [0] + np.cumsum([a + b for a, b in zip(new, old)]).tolist()
    q, kv = normal(gen, cq[-1], heads, 192), normal(gen, ck[-1], heads, 256)
    rot = normal(gen, ck[-1], 576)[:, 512:]                          # the dense copy's columns: strided rows
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    big = torch.full((cq[-1] + 2, heads, 128), 7.0, dtype=dtype, device="cuda")
    out = pskv.prefill_attn_expanded(q, kv, rot, dev(cq), cq, dev(ck), ck, 192 ** -0.5, out=big[1:-1],
                                     status=status)
    check_attention(out, expanded_reference(q, kv, rot, cq, ck, 192 ** -0.5), float(kv.abs().max()))
    assert (big[0] == 7).all() and (big[-1] == 7).all() and int(status[0]) == 0
    again = pskv.prefill_attn_expanded(q, kv, rot, dev(cq), cq, dev(ck), ck, 192 ** -0.5, out_dtype=dtype)
    assert torch.equal(out, again)


@pytest.mark.parametrize("new,old,heads", [
    ([600, 520, 700], [130, 0, 64], 40),                    # more blocks than clusters fit the GPU
    ([300] + [1, 0, 7, 33] * 10, [5] + [200, 0, 1, 90] * 10, 16),   # more rows than a warp's lanes
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_expanded_blocks_follow_one_another(new, old, heads, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(len(new))
    cq = [0] + np.cumsum(new).tolist()
    ck = [0] + np.cumsum([a + b for a, b in zip(new, old)]).tolist()
    q, kv, rot = normal(gen, cq[-1], heads, 192), normal(gen, ck[-1], heads, 256), normal(gen, ck[-1], 64)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = pskv.prefill_attn_expanded(q, kv, rot, dev(cq), cq, dev(ck), ck, 192 ** -0.5, out_dtype=dtype, status=status)
    check_attention(out, expanded_reference(q, kv, rot, cq, ck, 192 ** -0.5), float(kv.abs().max()))
    again = [pskv.prefill_attn_expanded(q, kv, rot, dev(cq), cq, dev(ck), ck, 192 ** -0.5, out_dtype=dtype)
             for _ in range(3)]
    assert all(torch.equal(out, o) for o in again) and int(status[0]) == 0


@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_expanded_scales_that_are_not_positive(scale):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    q, kv, rot = normal(gen, 200, 2, 192), normal(gen, 270, 2, 256), normal(gen, 270, 64)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out = pskv.prefill_attn_expanded(q, kv, rot, dev([0, 200]), [0, 200], dev([0, 270]), [0, 270], scale)
    check_attention(out, expanded_reference(q, kv, rot, [0, 200], [0, 270], scale), float(kv.abs().max()))


def test_expanded_growing_scores():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    n = 700
    q, kv, rot = normal(gen, n, 2, 192), normal(gen, n, 2, 256), normal(gen, n, 64)
    kv[..., :128] = (kv[..., :128].float() * torch.linspace(0.01, 2, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = pskv.prefill_attn_expanded(q, kv, rot, cu, [0, n], cu, [0, n], 1.0, out_dtype=torch.float32)
    ref = expanded_reference(q, kv, rot, [0, n], [0, n], 1.0)
    # |q.k| up to about 250: 192 * 2^-24 * 250 = 2.9e-3 of a score at worst
    assert (out.double() - ref).abs().max() <= 2 * (2.9e-3 + 2.0 ** -16) * float(kv.abs().max())
    assert float((out.double() - ref).norm() / ref.norm()) <= 2e-4


def test_expanded_rows_do_not_meet():
    """Another row's queries, keys and values may be anything: neighbours of a row that ends inside a tile."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    cq, ck = [0, 70, 100, 180], [0, 70, 130, 330]
    q, kv, rot = normal(gen, 180, 3, 192), normal(gen, 330, 3, 256), normal(gen, 330, 64)
    ref = expanded_reference(q, kv, rot, cq, ck, 0.07)
    top = float(kv.abs().max())
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q[70:100], kv[70:130], rot[70:130] = float("nan"), float("inf"), float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        out = pskv.prefill_attn_expanded(q, kv, rot, dev(cq), cq, dev(ck), ck, 0.07, out_dtype=dtype)
        for a, e in ((0, 70), (100, 180)):
            check_attention(out[a:e], ref[a:e], top)


def test_expanded_captured_and_on_two_streams():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cq, ck = [0, 300, 900], [0, 500, 1100]
    q, kv, rot = normal(gen, 900, 40, 192), normal(gen, 1100, 40, 256), normal(gen, 1100, 64)
    cu = dev(cq), dev(ck)
    call = lambda out, **kw: pskv.prefill_attn_expanded(q, kv, rot, cu[0], cq, cu[1], ck, 0.07, out=out, **kw)
    outs = [torch.empty(900, 40, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    call(outs[0])
    check_attention(outs[0], expanded_reference(q, kv, rot, cq, ck, 0.07), float(kv.abs().max()))
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):  # at once
        for s, o in zip(sides, outs[1:]):
            call(o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sides[0]):
        call(outs[1])
        call(outs[2])
    cu[0].copy_(dev([0, 250, 850]))  # other offsets within the host's blocks
    cu[1].copy_(dev([0, 410, 1010]))
    for _ in range(3):
        for o in outs[1:]:
            o.fill_(7.0)
        graph.replay()
    ref = expanded_reference(q, kv, rot, [0, 250, 850], [0, 410, 1010], 0.07)
    for o in outs[1:]:
        check_attention(o[:850], ref[:850], float(kv.abs().max()))
        assert (o[850:] == 7).all()


def test_expanded_offsets_that_disagree_are_skipped_and_flagged():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    q, kv, rot = normal(gen, 40, 2, 192), normal(gen, 60, 2, 256), normal(gen, 60, 64)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cq, ck = [0, 20, 40], [0, 30, 60]
    ref = expanded_reference(q, kv, rot, cq, ck, 0.1)
    for dq, dk in (([0, 20, 41], ck), ([0, 20, 40], [0, 30, 61]), ([0, 20, 40], [0, 30, 45])):
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        out = torch.full((40, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        pskv.prefill_attn_expanded(q, kv, rot, dev(dq), cq, dev(dk), ck, 0.1, out=out, status=status)
        assert int(status[0]) == pskv.PSKV_FAULT_BAD_LENGTH
        check_attention(out[:20], ref[:20], float(kv.abs().max()))
        assert (out[20:] == 7).all()


def test_compiled_and_python_calls_agree():
    """Calls of the plain form are compiled; host lengths of other types, host copies and options take
    the Python form."""
    c = LatentCase(17, [700, 65, 0], heads=24, tokens=2)
    ws = pskv.latent_workspace(c.layout, c.lens_host, 2, 24, table_stride=c.table.shape[1])
    plain = c.run(workspace=ws)
    with_arrays = pskv.decode_attn_latent(c.layout, c.q, c.table, c.lens, np.array(c.lens_host), c.scale)
    assert torch.equal(plain, with_arrays) and torch.equal(plain, c.run(workspace=ws, merge_group=8))
    assert torch.equal(plain, c.run())                                       # no workspace given
    one = c.run(num_splits=1)                                                # and none needed
    assert torch.equal(one, c.run(num_splits=1, workspace=ws)) and not one[2].any()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q, kv, rot = normal(gen, 90, 2, 192), normal(gen, 120, 2, 256), normal(gen, 120, 64)
    cu = dev([0, 30, 90]), dev([0, 50, 120])
    a = pskv.prefill_attn_expanded(q, kv, rot, cu[0], [0, 30, 90], cu[1], [0, 50, 120], 0.1)
    b = pskv.prefill_attn_expanded(q, kv, rot, cu[0], np.array([0, 30, 90]), cu[1], (0, 50, 120), 0.1)
    assert torch.equal(a, b)
    layout, ang = c.layout, torch.rand(800, 32, device="cuda")
    x, lease = normal(gen, 2, 576), dev([11, 2, 0])
    rows = dev([0, 1]), dev([650, 3])
    pools = []
    for host in (None, ([0, 1], [650, 3], [11, 2, 0])):
        qo = torch.empty(2, 5, 64, dtype=torch.bfloat16, device="cuda")
        pskv.kv_prep_append_latent(layout, x, *rows, c.table, lease, 1e-6, None, ang, ang, q=q[:2, :1, :64].expand(2, 5, 64),
                                   q_out=qo, host=host)
        pools.append((c.pool.clone(), qo))
    assert torch.equal(pools[0][0].view(torch.int16), pools[1][0].view(torch.int16)) and torch.equal(pools[0][1], pools[1][1])
    with pytest.raises(pskv.PskvError):
        pskv.decode_attn_latent(layout, c.q, c.table, c.lens, [700, 65, 1], c.scale, workspace=ws)
    with pytest.raises(ValueError):
        c.run(workspace=ws, out=plain[:2])
    with pytest.raises(TypeError):
        c.run(workspace=ws, out_dtype=torch.float16)


# ---- together ------------------------------------------------------------------------

def test_a_speculative_step_over_a_latent_cache():
    """A prompt through the expanded form, a drafted window through the absorbed form, and the drafts
    verified: both forms read what one page write left, and agree on the window."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    heads, dc, prompt, window, page, batch = 8, 512, 150, 4, 64, 2
    w_k = normal(gen, heads, 128, dc, scale=dc ** -0.5).float()         # key up-projection
    w_v = normal(gen, heads, 128, dc, scale=dc ** -0.5).float()
    n = prompt + window
    pages = -(-n // page)
    pool = torch.full((batch * pages, 1, page, dc + ROT), float("nan"), dtype=torch.bfloat16, device="cuda")
    layout = pskv.paged_kv_layout_create(pool, None)
    table = torch.randperm(batch * pages, generator=torch.Generator().manual_seed(0)).to(torch.int32).reshape(batch, pages).cuda()
    lease = torch.full((batch,), pages, dtype=torch.int32, device="cuda")
    angle = torch.arange(n, device="cuda").double()[:, None] * 1e4 ** (-torch.arange(32, device="cuda").double() / 32)
    x, q = normal(gen, batch, n, dc + ROT), normal(gen, batch, n, heads, 192)
    dense = torch.empty(batch, n, dc + ROT, dtype=torch.bfloat16, device="cuda")
    scale = 192 ** -0.5
    for lo, hi in ((0, prompt), (prompt, n)):                            # the prompt's chunk, then the window's
        rows = torch.arange(batch, dtype=torch.int32, device="cuda").repeat_interleave(hi - lo)
        pos = torch.arange(lo, hi, dtype=torch.int32, device="cuda").repeat(batch)
        qc, dc_rows = q[:, lo:hi].reshape(-1, heads, 192).contiguous(), torch.empty(rows.numel(), dc + ROT, dtype=torch.bfloat16, device="cuda")
        pskv.kv_prep_append_latent(layout, x[:, lo:hi].reshape(-1, dc + ROT).contiguous(), rows, pos, table, lease,
                                   1e-6, None, angle.cos().float(), angle.sin().float(), pairs="adjacent",
                                   q=qc[..., 128:], q_out=qc[..., 128:], dense=dc_rows)
        q[:, lo:hi] = qc.reshape(batch, hi - lo, heads, 192)
        dense[:, lo:hi] = dc_rows.reshape(batch, hi - lo, dc + ROT)
    c = dense[..., :dc].float()
    kv = torch.cat([torch.einsum("bnc,hdc->bnhd", c, w_k), torch.einsum("bnc,hdc->bnhd", c, w_v)], -1).to(torch.bfloat16)
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n
    full = pskv.prefill_attn_expanded(q.reshape(-1, heads, 192), kv.reshape(-1, heads, 256),
                                      dense.reshape(-1, dc + ROT)[:, dc:], cu, cu.cpu(), cu, cu.cpu(), scale)
    full = full.reshape(batch, n, heads, 128)[:, prompt:]
    qa = torch.cat([torch.einsum("bthd,hdc->bthc", q[:, prompt:, :, :128].float(), w_k).to(torch.bfloat16),
                    q[:, prompt:, :, 128:]], -1).contiguous()
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    lat = pskv.decode_attn_latent(layout, qa, table, lens, [n] * batch, scale, out_dtype=torch.float32)
    absorbed = torch.einsum("bthc,hdc->bthd", lat, w_v)
    # the expanded keys and values, the absorbed queries and both results are each rounded to bf16 once
    # or twice on the way: some 2^-8 of the outputs' size apiece
    assert float((absorbed - full.float()).norm() / full.float().norm()) <= 6 * HALF_BF16
    vocab = 1001
    head = torch.randn(vocab, heads * 128, generator=gen, device="cuda") * 0.3
    p = torch.softmax(absorbed.reshape(batch, window, -1) @ head.T, -1)
    qd = torch.softmax(p[:, :-1].log() + 0.3 * torch.randn(batch, window - 1, vocab, generator=gen, device="cuda"), -1)
    drafts = torch.multinomial(qd.reshape(-1, vocab), 1, generator=gen).reshape(batch, window - 1).to(torch.int32)
    tokens, accepted = pskv.verify_drafts(p.contiguous(), qd.contiguous(), drafts, torch.rand(batch, window, device="cuda", generator=gen))
    for b in range(batch):
        a = int(accepted[b])
        assert torch.equal(tokens[b, :a], drafts[b, :a]) and 0 <= int(tokens[b, a]) < vocab
        assert (tokens[b, a + 1:] == -1).all()
