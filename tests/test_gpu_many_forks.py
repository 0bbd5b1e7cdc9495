"""kv_fork_rows of as many forks as a call takes: right, refusals across the whole call, and no slower than the same forks
in several calls by more than the checks against each other cost."""
import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from tree_cases import i32

pytestmark = pytest.mark.gpu

MOST = 65535


def rows(n, layers, length, page=16):
    """One prompt over two pages, n empty rows and a page for each."""
    pools = torch.zeros(layers, n + 2, 1, page, 320, dtype=torch.bfloat16, device="cuda")
    pools[:, :2].normal_(generator=torch.Generator(device="cuda").manual_seed(n))
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    made = [pskv.paged_kv_layout_create(pools[k], None, status if k == 0 else None) for k in range(layers)]
    table, lens, leases = np.full((n + 1, 2), -1), np.zeros(n + 1), np.zeros(n + 1)
    table[0], lens[0], leases[0] = [0, 1], length, 2
    return pools, status, made, i32(table), i32(lens), i32(leases)


@pytest.mark.parametrize("n,layers,length", [(1025, 3, 23), (5000, 2, 31), (MOST, 2, 17), (MOST, 1, 32)])
def test_many_forks(n, layers, length):
    pools, status, made, table, lens, leases = rows(n, layers, length)
    perm = np.random.default_rng(n).permutation(n)
    pskv.kv_fork_rows(made, i32(np.zeros(n)), i32(1 + perm), i32(2 + np.arange(n)), table, lens, leases)
    rest = length - 16
    assert int(status[0]) == 0 and bool((lens == length).all()) and bool((leases[1:] == 2).all())
    want = np.zeros((n + 1, 2), np.int32)
    want[0, 1], want[1 + perm, 1] = 1, 2 + np.arange(n)
    if rest == 16:  # whole pages are shared
        want[1:, 1] = 1
        rest = 0
    assert np.array_equal(table.cpu().numpy(), want)
    assert bool((pools[:, 2:, 0, :rest] == pools[:, 1:2, 0, :rest]).all()) and not bool(pools[:, 2:, 0, rest:].any())


def test_refusals_across_a_whole_call():
    """Two forks far apart that name one row, and one whose row another reads."""
    pools, status, made, table, lens, leases = rows(MOST, 2, 20)
    dst = 1 + np.arange(MOST)
    dst[MOST - 1] = dst[3]
    src = np.zeros(MOST)
    src[40000] = dst[17]
    before = table.clone()
    pskv.kv_fork_rows(made, i32(src), i32(dst), i32(2 + np.arange(MOST)), table, lens, leases)
    gone = np.zeros(MOST, bool)
    gone[[3, 17, MOST - 1]] = True
    assert int(status[0]) == pskv.PSKV_FAULT_BAD_ROW
    got = lens.cpu().numpy()
    assert (got[dst[gone]] == 0).all() and torch.equal(table[4], before[4]) and torch.equal(table[18], before[18])
    want = np.where(src == 0, 20, 0)  # (row 18 was empty: so is the row that continues it)
    assert np.array_equal(got[dst[~gone]], want[~gone])
    filled = pools[:, 2:, 0, :4].flatten(2).any(-1).all(0).cpu().numpy()
    assert np.array_equal(filled, ~gone & (src == 0))


def test_one_call_and_sixteen_take_about_as_long():
    """(Each fork is compared with all others of its call: a sixteenth of the comparisons in the parts.)"""
    n, layers = MOST, 8
    pools, status, made, table, lens, leases = rows(n, layers, 23)
    src, dst, new = i32(np.zeros(n)), i32(1 + np.arange(n)), i32(2 + np.arange(n))

    def calls(parts):
        for k in range(parts):
            s = slice(k * n // parts, (k + 1) * n // parts)
            pskv.kv_fork_rows(made, src[s], dst[s], new[s], table, lens, leases)

    def ms(parts):
        best = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            calls(parts)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    ms(16)
    whole, parts = ms(1), ms(16)
    assert whole <= 6 * parts, (whole, parts)
