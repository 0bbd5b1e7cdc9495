"""sample_tokens on the GPU against its definition in whole numbers, and its probabilities against f64."""
import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from tree_cases import sample_reference

pytestmark = pytest.mark.gpu

FILTERS = [dict(), dict(top_k=5), dict(top_p=0.8), dict(min_p=0.05), dict(top_k=40, top_p=0.9),
           dict(top_k=300, top_p=0.99, min_p=0.001)]


def inputs(seed, batch, each, vocab, dtype, spread=2.5, lattice=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    l = spread * torch.randn(batch, each, vocab, generator=gen, device="cuda")
    if lattice:
        l = torch.round(l * lattice) / lattice  # many equal logits
    return l.to(dtype), torch.rand(batch, each, generator=gen, device="cuda")


def filters(batch, heat=True, top_k=0, top_p=1.0, min_p=0.0):
    """Values of each request around the given ones."""
    i = torch.arange(batch, device="cuda")
    out = {}
    if heat:
        out["temperature"] = 0.6 + 0.25 * (i % 5).float()
    if top_k:
        out["top_k"] = (top_k + i % 3).to(torch.int32)
    if top_p < 1:
        out["top_p"] = top_p - 0.03 * (i % 2).float()
    if min_p:
        out["min_p"] = min_p * (1.0 + i.float() % 3)
    return out


def check(logits, u, probs_dtype=None, **kw):
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    three = logits if logits.dim() == 3 else logits[:, None]
    u3 = None if u is None else u.reshape(three.shape[:2])
    probs = None if probs_dtype is None else torch.full(logits.shape, 7.0, dtype=probs_dtype, device="cuda")
    tokens = pskv.sample_tokens(logits, u, probs=probs, status=status, **kw)
    host = {k: None if v is None else v.tolist() for k, v in kw.items() if k in ("temperature", "top_k", "top_p", "min_p")}
    want, p = sample_reference(three, u3, **host)
    if u is not None:
        assert tokens.dtype == torch.int32 and tokens.shape == u.shape
        assert np.array_equal(tokens.cpu().numpy().reshape(want.shape), want)
    if probs is not None:
        # one rounding to f32 of W / S by a product of float pairs (another 2^-24 at most), then one to bf16
        half = 2.0 ** -23 if probs_dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -23
        got = probs.double().cpu().numpy().reshape(p.shape)
        assert (np.abs(got - p) <= half * p).all() and ((got == 0) == (p == 0)).all()
    return int(status[0])


@pytest.mark.parametrize("batch,each,vocab", [(1, 1, 1), (3, 1, 7), (2, 2, 33), (5, 1, 1000), (2, 3, 4099), (2, 1, 20001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", range(len(FILTERS)))
def test_matches_the_definition(batch, each, vocab, dtype, which):
    l, u = inputs(100 * vocab + which, batch, each, vocab, dtype)
    kind = [None, torch.float32, torch.bfloat16][which % 3]
    assert check(l, u, kind, **filters(batch, **FILTERS[which])) == 0


@pytest.mark.parametrize("vocab,dtype", [(131072, torch.float32), (131072, torch.bfloat16), (262147, torch.float32),
                                         (350000, torch.float32), (700001, torch.bfloat16)])
@pytest.mark.parametrize("which", [0, 2, 4, 5])
def test_large_vocabularies(vocab, dtype, which):
    l, u = inputs(vocab + which, 2, 1, vocab, dtype)
    assert check(l, u, torch.float32 if which == 4 else None, **filters(2, **FILTERS[which])) == 0


def test_the_largest_vocabulary():
    l, u = inputs(5, 1, 1, 1 << 22, torch.bfloat16)
    assert check(l, u, **filters(1, top_k=1000, top_p=0.9)) == 0


@pytest.mark.parametrize("lattice", [1, 4, 64])
@pytest.mark.parametrize("which", range(1, len(FILTERS)))
def test_equal_logits_go_by_index(lattice, which):
    l, u = inputs(lattice, 3, 1, 5000, torch.float32, lattice=lattice)
    assert check(l, u, torch.float32, **filters(3, **FILTERS[which])) == 0
    l = torch.zeros(3, 1, 5000, device="cuda")  # all equal
    assert check(l, u, torch.float32, **filters(3, **FILTERS[which])) == 0


@pytest.mark.parametrize("spread", [0.0003, 0.05, 40.0, 3000.0])
@pytest.mark.parametrize("which", [2, 4, 5])
def test_narrow_and_wide_logits(spread, which):
    l, u = inputs(3, 2, 1, 9001, torch.float32, spread=spread)
    assert check(l, u, torch.float32, **filters(2, **FILTERS[which])) == 0
    assert check(l - 1e4, u, **filters(2, **FILTERS[which])) == 0


def test_masked_logits_infinities_and_nans():
    l, u = inputs(4, 8, 1, 3001, torch.float32)
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    l[0, 0, 5:] = -inf
    l[1, 0, ::2] = nan
    l[2, 0, 17], l[2, 0, 2900] = inf, inf
    l[3, 0, :2999] = low
    l[4, 0] = -inf
    l[5, 0] = nan
    l[6, 0] = low
    l[7, 0, 0], l[7, 0, 1], l[7, 0, 2:] = torch.finfo(torch.float32).max, low, -inf
    for kw in FILTERS:
        assert check(l, u, torch.float32, **filters(8, **kw)) == pskv.PSKV_FAULT_EMPTY_ROW
    b = l.to(torch.bfloat16)
    assert check(b, u, torch.bfloat16, **filters(8, top_k=3, top_p=0.5)) == pskv.PSKV_FAULT_EMPTY_ROW


def test_settings_at_and_past_their_ends():
    l, u = inputs(6, 12, 1, 2000, torch.float32)
    inf, nan = float("inf"), float("nan")
    f = lambda *v: torch.tensor(v, dtype=torch.float32, device="cuda")
    heat = f(0.0, -1.0, nan, inf, 1e-45, 1e-38, 1e-30, 1e30, 0.5, 1.0, 2.0, 100.0)
    top_p = f(0.0, -1.0, nan, 1.0, 2.0, 1 - 2.0 ** -24, 2.0 ** -149, 1e-10, inf, -inf, 0.3, 0.999999)
    min_p = f(0.0, -1.0, nan, 1.0, 2.0, inf, -inf, 0.5, 1e-30, 1e-6, 0.1, 0.9)
    top_k = torch.tensor([0, -5, 1, 2000, 2001, 1999, 2 ** 31 - 1, -2 ** 31, 2, 3, 7, 1998], dtype=torch.int32, device="cuda")
    assert check(l, u, torch.float32, temperature=heat) == 0
    one = torch.ones(12, device="cuda")
    assert check(l, u, torch.float32, top_p=top_p) == 0
    assert check(l, u, torch.float32, top_k=top_k, temperature=one) == 0
    assert check(l, u, torch.float32, min_p=min_p) == 0
    for k in range(3):
        assert check(l, u, torch.float32, temperature=heat.roll(k), top_k=top_k.roll(5 * k), top_p=top_p.roll(7 * k),
                     min_p=min_p.roll(3 * k)) == 0


def test_the_ends_of_u():
    l, _ = inputs(7, 7, 1, 500, torch.float32)
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, -3.0, float("nan"), 2.0 ** -149, float("inf")], device="cuda")[:, None]
    assert check(l, u) == 0
    assert check(l, u, top_k=torch.full((7,), 3, dtype=torch.int32, device="cuda")) == 0


def test_draws_follow_the_distribution():
    """u over an even grid: each token is drawn in proportion to its probability, to one grid step."""
    l, _ = inputs(8, 1, 1, 50, torch.float32)
    n = 4096
    u = ((torch.arange(n, device="cuda") + 0.5) / n)[None]
    tokens = pskv.sample_tokens(l.expand(1, n, 50).contiguous(), u)
    many = torch.bincount(tokens[0].long(), minlength=50).double().cpu() / n
    assert (many - torch.softmax(l[0, 0].double().cpu(), -1)).abs().max() <= 1.5 / n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padded_rows_and_rows_off_16_bytes(dtype):
    l, u = inputs(9, 4, 3, 1003, dtype)
    for pad in (0, 1, 5, 61):
        wide = torch.full((4, 3, 1003 + pad), float("nan"), dtype=dtype, device="cuda")
        wide[..., :1003] = l
        assert check(wide[..., :1003], u, torch.float32, **filters(4, top_k=50, top_p=0.9)) == 0
    flat = torch.empty(l.numel() + 3, dtype=dtype, device="cuda")[3:].view(l.shape).copy_(l)
    assert check(flat, u, **filters(4, top_p=0.9)) == 0
    wide = torch.zeros(4, 6, 1003, dtype=dtype, device="cuda")
    wide[:, 3:4] = l[:, :1]
    assert check(wide[:, 3], u[:, 0].contiguous(), **filters(4, top_k=9)) == 0       # rows far apart, [batch, vocab]
    assert check(wide[:, 3:4], u[:, :1].contiguous(), **filters(4, top_k=9)) == 0


def test_only_probabilities():
    l, _ = inputs(10, 3, 2, 700, torch.bfloat16)
    probs = torch.empty(3, 2, 700, device="cuda")
    assert pskv.sample_tokens(l, None, probs=probs) is None
    assert check(l, None, torch.float32, **filters(3, top_k=20)) == 0
    # what verify_drafts takes: sums of one
    assert (probs.double().sum(-1) - 1).abs().max() < 1e-4


def test_far_rows():
    """Rows past 32 bits of elements."""
    rows, vocab = 5, 1000
    step = (1 << 31) // 2 + 8
    big = torch.empty(4 * step + vocab, dtype=torch.bfloat16, device="cuda")
    l, u = inputs(11, rows, 1, vocab, torch.bfloat16)
    view = torch.as_strided(big, (rows, vocab), (step, 1))
    view.copy_(l[:, 0])
    assert check(view, u[:, 0].contiguous(), **filters(rows, top_p=0.9)) == 0


def test_capture_streams_and_repeats():
    l, u = inputs(12, 4, 2, 5000, torch.float32)
    kw = filters(4, top_k=100, top_p=0.9)
    tokens, probs = torch.empty(4, 2, dtype=torch.int32, device="cuda"), torch.empty(l.shape, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pskv.sample_tokens(l, u, tokens=tokens, probs=probs, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        assert pskv.sample_tokens(l, u, tokens=tokens, probs=probs, **kw) is tokens
    host = {k: v.tolist() for k, v in kw.items()}
    for k in range(3):
        l.copy_(inputs(20 + k, 4, 2, 5000, torch.float32)[0])
        graph.replay()
        want, p = sample_reference(l, u, **host)
        assert np.array_equal(tokens.cpu().numpy(), want)
        first = probs.clone()
        graph.replay()
        assert torch.equal(first, probs)
    a = pskv.sample_tokens(l, u, stream=side, **kw)
    side.synchronize()
    assert np.array_equal(a.cpu().numpy(), want)


def test_python_refusals():
    l, u = inputs(13, 2, 2, 50, torch.float32)
    with pytest.raises(ValueError):
        pskv.sample_tokens(l, u[:, :1].contiguous())
    with pytest.raises(TypeError):
        pskv.sample_tokens(l.half(), u)
    with pytest.raises(TypeError):
        pskv.sample_tokens(l.cpu(), u)
    with pytest.raises(ValueError):
        pskv.sample_tokens(l.transpose(1, 2), u)
    with pytest.raises(ValueError):
        pskv.sample_tokens(l[:, :1].expand(2, 2, 50), u)
    with pytest.raises(ValueError):
        pskv.sample_tokens(torch.zeros(2, 3, 50, device="cuda")[:, :2], u)  # two steps from row to row
    with pytest.raises(ValueError):
        pskv.sample_tokens(l, u, temperature=torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        pskv.sample_tokens(l, u, top_k=torch.ones(2, device="cuda"))
    with pytest.raises(TypeError):
        pskv.sample_tokens(l, u, probs=torch.zeros(2, 2, 50, dtype=torch.float16, device="cuda"))
    with pytest.raises(pskv.PskvError):
        pskv.sample_tokens(l, None)
    with pytest.raises(pskv.PskvError):
        pskv.sample_tokens(l, None, tokens=torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
                           probs=torch.zeros(2, 2, 50, device="cuda"))
    with pytest.raises(ValueError):
        pskv.sample_tokens(l[0, 0], u[0, 0])


def test_top_k_past_the_tokens_with_weight():
    """More places than tokens that weigh anything: nothing is left out, min_p and top_p still count."""
    l, u = inputs(14, 4, 1, 3000, torch.float32, spread=1.0)
    l[:, :, 40:] -= 60.0  # expf(-60) is under 2^-41
    k = torch.tensor([41, 500, 2999, 40], dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(min_p=torch.full((4,), 0.05, device="cuda")), dict(top_p=torch.full((4,), 0.7, device="cuda")),
               dict(min_p=torch.full((4,), 0.02, device="cuda"), top_p=torch.full((4,), 0.9, device="cuda"))):
        assert check(l, u, torch.float32, top_k=k, **kw) == 0


@pytest.mark.parametrize("k,p,least", [(1500, 0.5, 0.0), (1500, 0.97, 0.01), (4000, 0.999, 0.0), (12000, 0.9, 0.001), (1020, 0.99, 0.0)])
def test_borders_behind_what_a_list_holds(k, p, least):
    """Flat rows whose kept tokens do not fit a list: borders by number and then by weight, draws over the whole row."""
    for dtype, lattice in ((torch.float32, None), (torch.bfloat16, None), (torch.float32, 8)):
        l, u = inputs(15 + k, 3, 1, 32001, dtype, spread=0.7, lattice=lattice)
        kw = dict(top_k=torch.tensor([k, k + 1, k + 7], dtype=torch.int32, device="cuda"), top_p=torch.full((3,), p, device="cuda"))
        if least:
            kw["min_p"] = torch.full((3,), least, device="cuda")
        assert check(l, u, torch.float32, **kw) == 0


def test_many_rows():
    """Batches that take clusters of eight, four, two and one."""
    for rows in (70, 100, 200, 700):
        l, u = inputs(rows, rows, 1, 600, torch.float32)
        assert check(l, u, **filters(rows, top_k=30, top_p=0.9)) == 0
        assert check(l, u, **filters(rows, top_p=0.95)) == 0


@pytest.mark.parametrize("rows", [76, 150, 303, 620])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", range(len(FILTERS)))
def test_batches_that_fill_the_chip(rows, dtype, which):
    """Rows that are read from memory again, off 16 bytes, many equal logits and masked ones, some at temperature 0."""
    l, u = inputs(rows + which, rows, 1, 1237, dtype, lattice=[None, 4, 2][which % 3])
    l = l[:, 0, 1:1236]
    l[:, 5::3] = -float("inf")
    l[3] = 0.5  # all equal
    l[4, 7:] = -float("inf")
    kw = filters(rows, **FILTERS[which])
    kw["temperature"][7::9] = 0.0
    assert check(l, u[:, 0].contiguous(), torch.float32 if which % 2 else None, **kw) == 0


@pytest.mark.parametrize("vocab,start,n", [(1000, 0, 1000), (1000, 1, 998), (4000, 700, 150), (32001, 9000, 700), (131072, 40000, 2000)])
@pytest.mark.parametrize("k,p", [(5, 1.0), (5, 0.5), (130, 1.0), (140, 0.9), (600, 1.0), (900, 0.7), (0, 0.3), (0, 0.999)])
@pytest.mark.parametrize("lattice", [None, 4])
def test_runs_of_allowed_tokens(vocab, start, n, k, p, lattice):
    """What is kept lies in a few warps' pieces; likelier tokens before many equal ones."""
    l, u = inputs(vocab + n + k, 3, 1, vocab, torch.float32, lattice=lattice)
    l[..., :start] = l[..., start + n:] = -float("inf")
    l[1, :, start:start + n] = torch.where(torch.arange(n, device="cuda") % 97 == 5, 9.0, 0.0)
    kw = {} if k == 0 else dict(top_k=torch.full((3,), k, dtype=torch.int32, device="cuda"))
    if p < 1:
        kw["top_p"] = torch.full((3,), p, device="cuda")
    assert check(l, u, torch.float32 if k % 2 else None, **kw) == 0


@pytest.mark.parametrize("vocab,start,n", [(600, 0, 600), (4000, 1500, 300), (40000, 7, 1000)])
@pytest.mark.parametrize("p", [0.9999, 0.999999, 0.99999994])
@pytest.mark.parametrize("above", [6.0, 15.0, 22.0])
def test_a_dominating_token_and_a_run_of_light_ones(vocab, start, n, p, above):
    """top-p's border among weights that its estimates do not tell apart."""
    l, u = inputs(vocab, 3, 1, vocab, torch.float32, spread=0.2)
    l[..., :start] = l[..., start + n:] = -float("inf")
    l[:, :, start + n // 2] = above
    l[2] = torch.round(l[2])
    kw = dict(top_p=torch.full((3,), p, device="cuda"))
    assert check(l, u, torch.float32, **kw) == 0
    assert check(l, u, top_k=torch.tensor([n // 2, n - 1, n + 5], dtype=torch.int32, device="cuda"), **kw) == 0


def test_top_k_that_keeps_all_with_weight_then_top_p():
    """The first search ends at once and the second begins: many times over, on a filled chip."""
    l, u = inputs(5, 76, 1, 1500, torch.float32)
    l[..., 100:] = -float("inf")
    kw = dict(top_k=torch.full((76,), 120, dtype=torch.int32, device="cuda"), top_p=torch.full((76,), 0.7, device="cuda"))
    first = pskv.sample_tokens(l, u, **kw)
    for _ in range(300):
        again = pskv.sample_tokens(l, u, **kw)
    assert torch.equal(first, again) and check(l, u, **kw) == 0


@pytest.mark.parametrize("rows,vocab,dtype", [(75, 131072, torch.bfloat16), (2, 1500001, torch.float32)])
def test_pieces_larger_than_shared_memory(rows, vocab, dtype):
    l, u = inputs(vocab, rows, 1, vocab, dtype)
    assert check(l, u, **filters(rows, top_k=300, top_p=0.99, min_p=0.001)) == 0
    assert check(l, u, **filters(rows, top_p=0.9)) == 0


def test_two_streams_at_once():
    """Calls that run beside each other on two streams, replayed and eager."""
    a, b = inputs(40, 24, 1, 40000, torch.float32), inputs(41, 40, 2, 9000, torch.bfloat16)
    kw = [filters(24, top_p=0.9), filters(40, top_k=60, top_p=0.8)]
    want = [sample_reference(*x, **{k: v.tolist() for k, v in w.items()})[0] for x, w in zip((a, b), kw)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (x, w) in enumerate(zip((a, b), kw)):
            got[i].append(pskv.sample_tokens(*x, stream=streams[i], **w))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(np.array_equal(t.cpu().numpy(), w) for t in g)


def test_python_forms_give_the_same(monkeypatch):
    """Without the compiled calls."""
    from paged_split_kv_attn_gb300 import _binding
    monkeypatch.setattr(_binding, "_calls", _binding._PythonCalls)
    l, u = inputs(42, 3, 2, 700, torch.float32)
    assert check(l, u, torch.bfloat16, **filters(3, top_k=20, top_p=0.9, min_p=0.01)) == 0
    assert check(l[:, 0], u[:, 0].contiguous()) == 0
