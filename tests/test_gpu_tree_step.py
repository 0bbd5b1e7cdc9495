"""Drafted trees over a latent cache, their walk, and the rows that are kept or forked, against plain references."""
import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import LatentCase, check_attention
from tree_cases import Cache, i32, i64, random_masks, sample_reference, walk_reference

pytestmark = pytest.mark.gpu


# ---- decode_attn_latent_tree ---------------------------------------------------------

def tree_reference(case, masks, hidden=None):
    """f64 attention over the keys before the window and those of the window that the masks hold."""
    T, out = case.tokens, torch.zeros(len(case.lens_host), case.tokens, case.heads, case.dc, dtype=torch.float64, device="cuda")
    for b, n in enumerate(case.lens_host):
        if n == 0:
            continue
        k = case.keys[b].double()
        s = torch.einsum("thd,kd->thk", case.q[b].double(), k) * case.scale
        for t in range(T):
            gone = [n - T + j for j in range(T) if j > t or not (int(masks[b, t]) >> j) & 1]
            s[t][:, gone] = -float("inf")
        if hidden is not None and hidden[b] is not None:
            s[:, :, hidden[b]] = -float("inf")
        w = torch.softmax(s, -1)
        w = torch.where(torch.isnan(w), torch.zeros_like(w), w)  # a token without any key
        out[b] = torch.einsum("thk,kd->thd", w, k[:, :case.dc])
    return out


def run_tree(case, masks, **kw):
    return pskv.decode_attn_latent_tree(case.layout, case.q, case.table, case.lens, case.lens_host, i64(masks), case.scale, **kw)


def check_tree(case, masks, faults=0, **kw):
    out = run_tree(case, masks, **kw)
    big = max(float(k.float().abs().max()) for k in case.keys if len(k))
    check_attention(out, tree_reference(case, masks), big)
    assert int(case.status[0]) == faults
    return out


@pytest.mark.parametrize("lens,tokens,heads,dc,page", [
    ([8], 8, 16, 512, 64), ([1], 1, 5, 256, 64), ([700, 33], 8, 32, 512, 64), ([129, 0, 300], 5, 16, 256, 16),
    ([64, 65, 127, 128, 191], 64, 3, 512, 64), ([2000, 40], 33, 8, 512, 256), ([515], 64, 128, 256, 48),
    ([5000, 100, 64], 16, 20, 512, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tree_matches_f64(lens, tokens, heads, dc, page, dtype):
    case = LatentCase(sum(lens) + tokens, lens, dc, page, heads, tokens)
    masks = random_masks(np.random.default_rng(tokens), len(lens), tokens, roots=0.1)
    check_tree(case, masks, out_dtype=dtype)


@pytest.mark.parametrize("splits", [1, 2, 7, 64])
def test_windows_at_every_place_of_a_tile(splits):
    """Windows that begin and end at every sixteenth key, across tiles and pieces."""
    for n in list(range(200, 456, 16)) + [255, 256, 257, 383, 384, 385]:
        case = LatentCase(n, [n, 640], 256, 64, 8, 40)
        masks = random_masks(np.random.default_rng(n), 2, 40, roots=0.2)
        check_tree(case, masks, num_splits=splits, out_dtype=torch.float32)


@pytest.mark.parametrize("splits", [0, 1, 5])
def test_a_chain_is_the_causal_window(splits):
    case = LatentCase(3, [900, 77, 1500], 512, 64, 24, 7)
    chain = np.tile((np.uint64(2) << np.arange(7, dtype=np.uint64)) - np.uint64(1), (3, 1))
    for dtype in (torch.bfloat16, torch.float32):
        assert torch.equal(run_tree(case, chain, num_splits=splits, out_dtype=dtype),
                           case.run(num_splits=splits, out_dtype=dtype))


def test_bad_masks_are_flagged():
    """A later bit is ignored, a missing own bit leaves the token without itself, nothing at all gives zeros."""
    case = LatentCase(4, [300, 4], 512, 64, 8, 4)
    masks = random_masks(np.random.default_rng(1), 2, 4)
    masks[0, 1] |= np.uint64(1 << 3 | 1 << 40)
    check_tree(case, masks, pskv.PSKV_FAULT_BAD_MASK, out_dtype=torch.float32)
    case.status.zero_()
    masks[0, 1], masks[0, 2] = 1, 2
    check_tree(case, masks, pskv.PSKV_FAULT_BAD_MASK, out_dtype=torch.float32)
    case.status.zero_()
    masks[1, 0] = 0  # the row's first key: no other before it
    out = check_tree(case, masks, pskv.PSKV_FAULT_BAD_MASK | pskv.PSKV_FAULT_EMPTY_ROW, out_dtype=torch.float32)
    assert (out[1, 0] == 0).all()


def test_tree_skips_bad_pages():
    case = LatentCase(5, [640, 300], 512, 64, 8, 6)
    masks = random_masks(np.random.default_rng(2), 2, 6)
    case.table[0, 9], case.table[1, 1] = -3, 1 << 30  # the window's own page, and one before it
    hidden = [torch.zeros(640, dtype=torch.bool, device="cuda"), torch.zeros(300, dtype=torch.bool, device="cuda")]
    hidden[0][576:], hidden[1][64:128] = True, True
    out = run_tree(case, masks, out_dtype=torch.float32)
    check_attention(out, tree_reference(case, masks, hidden), 6.0)
    assert int(case.status[0]) == pskv.PSKV_FAULT_BAD_PAGE


def test_tree_workspaces_options_and_capture():
    case = LatentCase(6, [4000, 900], 512, 256, 32, 9)
    masks = i64(random_masks(np.random.default_rng(3), 2, 9))
    call = lambda **kw: pskv.decode_attn_latent_tree(case.layout, case.q, case.table, case.lens, case.lens_host, masks,
                                                     case.scale, **kw)
    want = call()
    ws = pskv.latent_workspace(case.layout, case.lens_host, 9, 32)
    assert torch.equal(call(workspace=ws), want)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    assert torch.equal(call(events=(begin, end), merge_group=4), want)
    end.synchronize()
    assert begin.elapsed_time(end) > 0
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out=out, workspace=ws)
    masks.copy_(i64(random_masks(np.random.default_rng(4), 2, 9)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call()) and not torch.equal(out, want)


def test_tree_refusals():
    case = LatentCase(7, [100, 50], 256, 64, 8, 4)
    masks = random_masks(np.random.default_rng(5), 2, 4)
    with pytest.raises(ValueError):
        run_tree(case, masks[:, :3])
    with pytest.raises(TypeError):
        pskv.decode_attn_latent_tree(case.layout, case.q, case.table, case.lens, case.lens_host, i32([[1] * 4] * 2), case.scale)
    with pytest.raises(TypeError):
        pskv.decode_attn_latent_tree(case.layout, case.q, case.table, case.lens, case.lens_host, None, case.scale)
    with pytest.raises(pskv.PskvError):
        pskv.decode_attn_latent_tree(case.layout, case.q, case.table, case.lens, [100, 3], i64(masks), case.scale)


# ---- verify_tree -----------------------------------------------------------------------

@pytest.mark.parametrize("batch,T,words", [(1, 1, 1), (1, 8, 2), (7, 5, 1), (64, 64, 2), (33, 33, 1), (5, 64, 1), (200, 17, 3), (9, 32, 4)])
def test_walk_matches_the_definition(batch, T, words):
    rng = np.random.default_rng(batch + T)
    for chain in (False, True):
        masks = random_masks(rng, batch, T, roots=0.05)
        if chain:
            masks = np.tile(~np.uint64(0) >> (np.uint64(63) - np.arange(T, dtype=np.uint64)), (batch, 1))
        drafts, sampled = rng.integers(0, words, (batch, T)), rng.integers(0, words, (batch, T))
        sampled[rng.random((batch, T)) < 0.05] = -1
        drafts[rng.random((batch, T)) < 0.05] = -1
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        got = pskv.verify_tree(i32(drafts), i64(masks), i32(sampled), status=status)
        for g, w in zip(got, walk_reference(drafts, masks, sampled)):
            assert np.array_equal(g.cpu().numpy(), w)
        assert int(status[0]) == 0


def test_walk_of_bad_masks():
    rng = np.random.default_rng(1)
    masks = random_masks(rng, 3, 9)
    masks[0, 4] |= np.uint64(1 << 8)
    masks[1, 3] = 0
    masks[2, 2] = np.uint64(1)  # without itself: its parent is token 0 all the same
    drafts = sampled = np.zeros((3, 9), np.int64)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = pskv.verify_tree(i32(drafts), i64(masks), i32(sampled), status=status)
    for g, w in zip(got, walk_reference(drafts, masks, sampled)):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int(status[0]) == pskv.PSKV_FAULT_BAD_MASK


def test_walk_refusals_and_given_outputs():
    masks = random_masks(np.random.default_rng(2), 2, 6)
    d, s = i32(np.zeros((2, 6))), i32(np.zeros((2, 6)))
    outs = [torch.empty(2, 6, dtype=torch.int32, device="cuda"), torch.empty(2, 6, dtype=torch.int32, device="cuda"),
            torch.empty(2, dtype=torch.int32, device="cuda")]
    got = pskv.verify_tree(d, i64(masks), s, *outs)
    assert all(a is b for a, b in zip(got, outs))
    with pytest.raises(ValueError):
        pskv.verify_tree(d, i64(masks), s[:, :5].contiguous())
    with pytest.raises(ValueError):
        pskv.verify_tree(d[:, ::2], i64(masks[:, :3]), s[:, ::2])
    with pytest.raises(TypeError):
        pskv.verify_tree(d, i64(masks).int(), s)
    with pytest.raises(pskv.PskvError):
        z = torch.zeros(1, 65, dtype=torch.int32, device="cuda")
        pskv.verify_tree(z, torch.zeros(1, 65, dtype=torch.int64, device="cuda"), z)


# ---- kv_keep_tokens ----------------------------------------------------------------------

def keep_reference(c, pools, lens, path, kept, T):
    """Rows moved one after another in the host's copies; new lengths."""
    out = np.array(lens)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        w0 = n - T
        for i in range(kept[b]):
            s, d = w0 + path[b, i], w0 + i
            for p in pools:
                p[:, c.table[b, d // c.page], :, d % c.page] = p[:, c.table[b, s // c.page], :, s % c.page].clone()
        out[b] = w0 + kept[b]
    return out


def random_paths(rng, batch, T):
    kept = rng.integers(0, T + 1, batch)
    path = rng.integers(-5, 100, (batch, T))
    for b in range(batch):
        path[b, :kept[b]] = np.sort(rng.choice(T, kept[b], replace=False))
    return path.astype(np.int32), kept.astype(np.int32)


def equal(pools, want):
    return all(torch.equal(a, b) for a, b in zip(pools, want))


@pytest.mark.parametrize("kind", list(Cache.SHAPES))
@pytest.mark.parametrize("T,layers", [(1, 1), (2, 3), (17, 2), (64, 1)])
def test_keep_moves_the_rows(kind, T, layers):
    rng = np.random.default_rng(T)
    lens = [T, T + 1, 0, T + 63, 300 + T, 256]
    c = Cache(T, kind, lens, layers)
    path, kept = random_paths(rng, len(lens), T)
    want = c.host()
    new = keep_reference(c, want, lens, path, kept, T)
    got = pskv.kv_keep_tokens(c.layouts, c.dev_table, c.dev_lens, i32(path), i32(kept))
    assert np.array_equal(got.cpu().numpy(), new) and equal(c.pools, want) and c.faults() == 0
    assert np.array_equal(c.dev_lens.cpu().numpy(), lens)


def test_keep_of_one_layout_and_given_lengths():
    c = Cache(1, "latent512", [90, 400])
    path, kept = random_paths(np.random.default_rng(1), 2, 20)
    want = c.host()
    new = keep_reference(c, want, [90, 400], path, kept, 20)
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    dev_path, dev_kept = i32(path), i32(kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert pskv.kv_keep_tokens(c.layouts[0], c.dev_table, c.dev_lens, dev_path, dev_kept, new_lens=lens, stream=side) is lens
    side.synchronize()
    assert np.array_equal(lens.cpu().numpy(), new) and equal(c.pools, want)


class _Only:
    """Some rows of a cache."""

    def __init__(self, c, rows):
        self.table, self.page = c.table[rows], c.page


def test_keep_leaves_refused_rows():
    T, lens = 8, [100, 100, 100, 100, 100, 100, 7, 5000, -1, 100, 100]
    c = Cache(2, "split256", [100] * len(lens), layers=2)
    path = np.tile(np.array([0, 2, 4, 5, 6, 7, 9, 9], np.int32), (len(lens), 1))
    kept = np.full(len(lens), 4, np.int32)
    path[0, 1] = 0            # not going up
    path[1, 3] = 8            # past the window
    path[2, 0] = -1
    kept[3], kept[4] = 9, -1
    c.table[5, 1] = 1 << 20   # (keys 92 .. 99 lie in the second page)
    want = c.host()
    new = np.array(lens, np.int32)
    new[9:] = keep_reference(_Only(c, [9, 10]), want, [100, 100], path[9:], kept[9:], T)
    got = pskv.kv_keep_tokens(c.layouts, i32(c.table), i32(lens), i32(path), i32(kept))
    assert np.array_equal(got.cpu().numpy(), new) and equal(c.pools, want)
    assert c.faults() == pskv.PSKV_FAULT_BAD_PATH | pskv.PSKV_FAULT_BAD_LENGTH | pskv.PSKV_FAULT_BAD_PAGE


def test_keep_capture():
    c = Cache(3, "split512", [300, 280], layers=2)
    path, kept = i32([[0, 3, 5, 6, -1, -1, -1, -1]] * 2), i32([4, 2])
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pskv.kv_keep_tokens(c.layouts, c.dev_table, c.dev_lens, path, kept, new_lens=lens)
    want = c.host()
    for _ in range(2):  # twice: the second pass moves what the first one left
        new = keep_reference(c, want, [300, 280], path.cpu().numpy(), [4, 2], 8)
        graph.replay()
    torch.cuda.synchronize()
    assert equal(c.pools, want) and np.array_equal(lens.cpu().numpy(), new)


def test_keep_refusals():
    c, other = Cache(4, "latent512", [90, 90]), Cache(4, "latent256", [90, 90])
    path, kept = i32(np.zeros((2, 4))), i32([1, 1])
    with pytest.raises(pskv.PskvError):  # layers of two kinds
        pskv.kv_keep_tokens([c.layouts[0], other.layouts[0]], c.dev_table, c.dev_lens, path, kept)
    with pytest.raises(pskv.PskvError):
        pskv.kv_keep_tokens([], c.dev_table, c.dev_lens, path, kept)
    with pytest.raises(pskv.PskvError):
        pskv.kv_keep_tokens([c.layouts[0]] * 129, c.dev_table, c.dev_lens, path, kept)
    with pytest.raises(pskv.PskvError):  # in place
        pskv.kv_keep_tokens(c.layouts, c.dev_table, c.dev_lens, path, kept, new_lens=c.dev_lens)
    with pytest.raises(pskv.PskvError):
        pskv.kv_keep_tokens(c.layouts, c.dev_table, c.dev_lens, path, kept, new_lens=kept)
    with pytest.raises(ValueError):
        pskv.kv_keep_tokens(c.layouts, c.dev_table, c.dev_lens, path, i32([1]))
    with pytest.raises(TypeError):
        pskv.kv_keep_tokens(c.layouts, c.dev_table, c.dev_lens.long(), path, kept)
    layout = c.layouts[0]
    layout.close()
    with pytest.raises((pskv.PskvError, ValueError)):
        pskv.kv_keep_tokens(layout, c.dev_table, c.dev_lens, path, kept)


# ---- kv_fork_rows --------------------------------------------------------------------------

def fork_reference(c, pools, src, dst, new):
    """Forks one after another on the host's table, lengths and leases (changed in place)."""
    for i, (s, d) in enumerate(zip(src, dst)):
        n = int(c.lens[s])
        whole, rest = divmod(n, c.page)
        c.table[d, :whole] = c.table[s, :whole]
        if rest:
            for p in pools:
                p[:, new[i], :, :rest] = p[:, c.table[s, whole], :, :rest].clone()
            c.table[d, whole] = new[i]
        c.lens[d], c.leases[d] = n, whole + (rest > 0)


def check_fork(c, src, dst, new, want_faults=0, done=None):
    want = c.host()
    every = range(len(src)) if done is None else done
    pskv.kv_fork_rows(c.layouts, i32(src), i32(dst), i32(new), c.dev_table, c.dev_lens, c.dev_leases)
    fork_reference(c, want, [src[i] for i in every], [dst[i] for i in every], [new[i] for i in every])
    assert equal(c.pools, want) and c.faults() == want_faults
    assert np.array_equal(c.dev_table.cpu().numpy(), c.table)
    assert np.array_equal(c.dev_lens.cpu().numpy(), c.lens) and np.array_equal(c.dev_leases.cpu().numpy(), c.leases)


@pytest.mark.parametrize("kind", list(Cache.SHAPES))
@pytest.mark.parametrize("layers", [1, 3])
def test_forks_share_pages_and_copy_the_last(kind, layers):
    page = Cache.SHAPES[kind][3]
    lens = [1, page - 1, page, page + 1, 3 * page + 7, 0, 0, 0, 0, 0, 0, 0, 0, 0]
    c = Cache(layers, kind, lens, layers, stride=5, spare=9)
    src, dst = [0, 1, 2, 3, 4, 4, 4, 5], [13, 6, 7, 8, 9, 12, 10, 11]
    new = c.spare[:8].tolist()
    new[2] = new[7] = -99  # keys that fill their pages, or none: not looked at
    check_fork(c, src, dst, new)


def test_forks_over_rows_that_held_keys():
    """A row that is written again: entries past its pages stay."""
    c = Cache(5, "split256", [100, 700, 130], spare=3)
    check_fork(c, [0], [1], c.spare[:1].tolist())
    assert c.table[1, 2] != -7  # (what it held)
    check_fork(c, [1], [2], c.spare[1:2].tolist())


def test_forks_refused():
    page = 64
    c = Cache(6, "latent512", [100, 200, 300, 64, 90, 80, 70, 60, 50, 40, 30, 64], stride=5, spare=12, layers=2)
    new = c.spare[:9].tolist()
    # of each: out of range; itself; two that name one row; a row that another fork reads
    src = [-1, 12, 0, 1, 0, 0, 1, 3, 11]
    dst = [5, 6, 12, 1, 7, 7, 0, 8, 9]
    check_fork(c, src, dst, new, pskv.PSKV_FAULT_BAD_ROW, done=[7, 8])
    c.status.zero_()
    bad = c.dev_lens.clone(), c.dev_leases.clone(), c.dev_table.clone()
    for what, fault in [("lens", pskv.PSKV_FAULT_BAD_LENGTH), ("lens-", pskv.PSKV_FAULT_BAD_LENGTH),
                        ("lease", pskv.PSKV_FAULT_PAST_PAGES), ("lease+", pskv.PSKV_FAULT_PAST_PAGES),
                        ("page", pskv.PSKV_FAULT_BAD_PAGE), ("new", pskv.PSKV_FAULT_BAD_PAGE),
                        ("same", pskv.PSKV_FAULT_BAD_PAGE)]:
        page_new = new[0]
        if what == "lens":
            c.dev_lens[2] = 5 * page + 1
        if what == "lens-":
            c.dev_lens[2] = -1
        if what == "lease":
            c.dev_leases[2] = 4
        if what == "lease+":
            c.dev_leases[2] = 6
        if what == "page":
            c.dev_table[2, 4] = len(c.pools[0][0])
        if what == "new":
            page_new = -1
        if what == "same":
            page_new = int(c.dev_table[2, 4])
        before = [x.clone() for x in (*c.pools, c.dev_table, c.dev_lens, c.dev_leases)]
        pskv.kv_fork_rows(c.layouts, i32([2]), i32([4]), i32([page_new]), c.dev_table, c.dev_lens, c.dev_leases)
        assert all(torch.equal(a, b) for a, b in zip(before, (*c.pools, c.dev_table, c.dev_lens, c.dev_leases)))
        assert c.faults() == fault
        c.status.zero_()
        for t, b in zip((c.dev_lens, c.dev_leases, c.dev_table), bad):
            t.copy_(b)


def test_many_forks_of_one_row():
    c = Cache(7, "latent256", [1000] + [0] * 300, spare=300)
    check_fork(c, [0] * 300, list(range(300, 0, -1)), c.spare[:300].tolist())


def test_fork_capture_and_refusals():
    c = Cache(8, "f32", [90, 0, 0], spare=2)
    src, dst, new = i32([0, 0]), i32([1, 2]), i32(c.spare[:2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pskv.kv_fork_rows(c.layouts[0], src, dst, new, c.dev_table, c.dev_lens, c.dev_leases)
    want = c.host()
    fork_reference(c, want, [0, 0], [1, 2], c.spare[:2])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert equal(c.pools, want) and np.array_equal(c.dev_table.cpu().numpy(), c.table)
    pskv.kv_fork_rows(c.layouts, src[:0], dst[:0], new[:0], c.dev_table, c.dev_lens, c.dev_leases)  # none
    with pytest.raises(ValueError):
        pskv.kv_fork_rows(c.layouts, src, dst[:1].contiguous(), new, c.dev_table, c.dev_lens, c.dev_leases)
    with pytest.raises(TypeError):
        pskv.kv_fork_rows(c.layouts, src.long(), dst, new, c.dev_table, c.dev_lens, c.dev_leases)
    with pytest.raises(ValueError):
        pskv.kv_fork_rows(c.layouts, src, dst, new, c.dev_table, c.dev_lens[:2], c.dev_leases)
    assert c.faults() == 0


# ---- together --------------------------------------------------------------------------------

def test_a_step_of_drafted_trees_over_forked_rows():
    """A prompt's row is forked, each fork's tree attended, sampled at its tokens, judged, kept; then the next
    token attends what a plain cache of the kept rows holds."""
    heads, T, forks, vocab, prompt = 16, 6, 3, 500, 150
    rng, gen = np.random.default_rng(9), torch.Generator(device="cuda").manual_seed(9)
    c = Cache(9, "latent512", [prompt] + [0] * forks, spare=4 * forks, stride=4)
    keys = c.pools[0][0][torch.from_numpy(c.table[0].astype(np.int64)).cuda()[:3], 0].reshape(-1, 576)[:prompt].clone()
    pskv.kv_fork_rows(c.layouts, i32([0] * forks), i32([1, 2, 3]), i32(c.spare[:forks]), c.dev_table, c.dev_lens, c.dev_leases)
    # the forks' windows go behind the prompt (a page more each)
    table = c.dev_table.clone()
    table[1:, 3] = i32(c.spare[forks:2 * forks])
    x = torch.randn(forks * T, 576, generator=gen, device="cuda").to(torch.bfloat16)
    rows, pos = np.repeat(np.arange(1, forks + 1), T), np.tile(prompt + np.arange(T), forks)
    cos, sin = torch.ones(256, 32, device="cuda"), torch.zeros(256, 32, device="cuda")
    dense = torch.empty_like(x)
    pskv.kv_prep_append_latent(c.layouts[0], x, i32(rows), i32(pos), table, i32([3, 4, 4, 4]), 1e-6, None, cos, sin, dense=dense)
    masks = random_masks(rng, forks, T)
    lens = [0] + [prompt + T] * forks
    q = torch.randn(forks + 1, T, heads, 576, generator=gen, device="cuda").to(torch.bfloat16)
    all_masks = np.concatenate([np.tile(np.uint64(1) << np.arange(T, dtype=np.uint64), (1, 1)), masks])
    out = pskv.decode_attn_latent_tree(c.layouts[0], q, table, i32(lens), lens, i64(all_masks), 0.07)
    logits = torch.randn(heads * 512, vocab, generator=gen, device="cuda") * 0.02
    logits = (out.flatten(2).float() @ logits).contiguous()
    u = torch.rand(forks + 1, T, generator=gen, device="cuda")
    kw = dict(top_k=i32([20] * (forks + 1)), top_p=torch.full((forks + 1,), 0.9, device="cuda"))
    sampled = pskv.sample_tokens(logits, u, **kw)
    assert np.array_equal(sampled.cpu().numpy(), sample_reference(logits, u, top_k=[20] * 4, top_p=[float(np.float32(0.9))] * 4)[0])
    # drafts that follow the target at some places
    says, drafts = sampled.cpu().numpy(), rng.integers(0, vocab, (forks + 1, T))
    for b in range(1, forks + 1):
        for t in range(1, T):
            if rng.random() < 0.7:
                drafts[b, t] = says[b, (int(all_masks[b, t]) & ((1 << t) - 1)).bit_length() - 1]
    tokens, path, kept = pskv.verify_tree(i32(drafts), i64(all_masks), sampled)
    for g, w in zip((tokens, path, kept), walk_reference(drafts, all_masks, says)):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int(kept[1:].max()) > 1
    new_lens = pskv.kv_keep_tokens(c.layouts, table, i32(lens), path, kept)
    host_lens = new_lens.tolist()
    assert host_lens == [0] + [prompt + k for k in kept[1:].tolist()] and c.faults() == 0
    q1 = torch.randn(forks + 1, 1, heads, 576, generator=gen, device="cuda").to(torch.bfloat16)
    out = pskv.decode_attn_latent(c.layouts[0], q1, table, new_lens, host_lens, 0.07, out_dtype=torch.float32)
    for b in range(1, forks + 1):
        mine = torch.cat([keys, dense[(b - 1) * T + path[b, :int(kept[b])].long()]]).double()
        w = torch.softmax(q1[b, 0].double() @ mine.T * 0.07, -1)
        ref = (w @ mine[:, :512])[None, None]
        check_attention(out[b:b + 1], ref, float(mine.abs().max()))


def test_python_forms_give_the_same(monkeypatch):
    """Without the compiled calls: the step above, the chain, the refusals."""
    from paged_split_kv_attn_gb300 import _binding
    monkeypatch.setattr(_binding, "_calls", _binding._PythonCalls)
    test_a_step_of_drafted_trees_over_forked_rows()
    test_a_chain_is_the_causal_window(0)
    test_tree_refusals()
    test_walk_refusals_and_given_outputs()
    test_keep_refusals()
    test_fork_capture_and_refusals()


def test_uint64_masks():
    case = LatentCase(8, [200], 256, 64, 8, 5)
    masks = random_masks(np.random.default_rng(6), 1, 5)
    unsigned = torch.from_numpy(masks).cuda()
    assert unsigned.dtype == torch.uint64
    out = pskv.decode_attn_latent_tree(case.layout, case.q, case.table, case.lens, case.lens_host, unsigned, case.scale)
    assert torch.equal(out, run_tree(case, masks))
    d = i32(np.zeros((1, 5)))
    assert all(torch.equal(a, b) for a, b in zip(pskv.verify_tree(d, unsigned, d), pskv.verify_tree(d, i64(masks), d)))


def test_workspaces_shared_by_two_graphs():
    """Two captured calls that use one workspace, replayed one after another in either order."""
    a, b = LatentCase(9, [3000], 512, 256, 16, 6), LatentCase(10, [2500, 700], 512, 256, 16, 4)
    need = max(pskv.decode_attn_latent_workspace_bytes(c.layout, c.lens_host, c.table.shape[1], c.tokens, c.heads) for c in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    calls = []
    for c in (a, b):
        masks = i64(random_masks(np.random.default_rng(c.tokens), len(c.lens_host), c.tokens))
        out = torch.empty(len(c.lens_host), c.tokens, 16, 512, dtype=torch.bfloat16, device="cuda")
        args = (c.layout, c.q, c.table, c.lens, c.lens_host, masks, c.scale)
        want = pskv.decode_attn_latent_tree(*args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pskv.decode_attn_latent_tree(*args, workspace=ws, out=out)
        calls.append((graph, out, want))
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for k in order:
            calls[k][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(calls[k][1], calls[k][2]) for k in order)


def test_keep_and_fork_far_into_a_pool():
    """Pages whose rows lie past 2^31 elements of a region."""
    heads, page, d = 16, 64, 256
    pages = (1 << 31) // (heads * page * d) + 9
    k = torch.zeros(pages, heads, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    layout = pskv.paged_kv_layout_create(k, v)
    gen = torch.Generator(device="cuda").manual_seed(1)
    far = [pages - 2, pages - 3, pages - 5]
    for p in far[:2]:
        k[p] = torch.randn(k[p].shape, generator=gen, device="cuda").to(torch.bfloat16)
        v[p] = torch.randn(k[p].shape, generator=gen, device="cuda").to(torch.bfloat16)
    table, lens, leases = i32([far[:2], [-1, -1]]), i32([100, 0]), i32([2, 0])
    pskv.kv_fork_rows(layout, i32([0]), i32([1]), i32(far[2:]), table, lens, leases)
    assert table.tolist() == [far[:2], [far[0], far[2]]] and lens.tolist() == [100, 100]
    for pool in (k, v):
        assert torch.equal(pool[far[2], :, :36], pool[far[1], :, :36]) and not pool[far[2], :, 36:].any()
    want = [torch.cat([pool[far[0]], pool[far[2]]], 1)[:, [90, 93, 99]].clone() for pool in (k, v)]
    new = pskv.kv_keep_tokens(layout, table, lens, i32([[0] * 10, [0, 3, 9] + [-1] * 7]), i32([0, 3]))
    assert new.tolist() == [90, 93]
    for pool, w in zip((k, v), want):
        assert torch.equal(pool[far[2], :, 26:29], w)
