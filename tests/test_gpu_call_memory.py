"""Memory that a call makes for itself (outputs, scratch) belongs to the stream it runs on: nothing of
the current stream meets it, before the call or after."""
import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
import workloads as W
from gpu_cases import DevCase, i32, to_dev
from latent_cases import LatentCase, normal

pytestmark = pytest.mark.gpu

PAUSE = 50_000_000  # clock cycles: some 25 ms


def calls():
    """name -> call(stream): its outputs.  Inputs are kept here, past every call."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(31)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    c = LatentCase(31, [3000, 700])
    q, kv, rot = normal(gen, 90, 2, 192), normal(gen, 120, 2, 256), normal(gen, 120, 64)
    cu = dev([0, 30, 90]), dev([0, 50, 120])
    target = torch.softmax(torch.randn(5, 3, 901, generator=gen, device="cuda"), -1)
    drafts, u = torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.rand(5, 3, generator=gen, device="cuda")
    d = DevCase(W.make_paged_case(0, [1000, 300], dtype="bf16", **W.GLOBAL_SHAPE))
    pcu = np.array([0, 40, 80], np.int32)
    pcu_dev = i32(pcu)
    qp = to_dev(W.bf16_bits(np.random.default_rng(5).standard_normal((80, 32, 512), dtype=np.float32)), "bf16")
    qw = to_dev(W.window_queries(d.case, 2), "bf16")
    m, l, o = torch.zeros(9, 3, device="cuda"), torch.ones(9, 3, device="cuda"), torch.randn(9, 3, 512, generator=gen, device="cuda")
    scale = d.case.scale
    return {
        "decode_attn_latent": lambda s: [c.run(stream=s)],
        "decode_attn_latent, Python": lambda s: [c.run(stream=s, merge_group=8)],
        "decode_attn_latent, one piece": lambda s: [c.run(stream=s, num_splits=1)],
        "prefill_attn_expanded": lambda s: [pskv.prefill_attn_expanded(q, kv, rot, cu[0], [0, 30, 90], cu[1], [0, 50, 120], 0.1, stream=s)],
        "prefill_attn_expanded, Python": lambda s: [pskv.prefill_attn_expanded(q, kv, rot, cu[0], (0, 30, 90), cu[1], (0, 50, 120), 0.1, stream=s)],
        "verify_drafts": lambda s: list(pskv.verify_drafts(target, None, drafts, u, stream=s)),
        "decode_attn_splitkv": lambda s: [d.decode(stream=s, num_splits=4)],
        "decode_attn_multirow": lambda s: [pskv.decode_attn_multirow(d.layout, qw, d.tables, d.lens, d.case.seq_lens, scale, num_splits=4, stream=s)],
        "prefill_attn_paged": lambda s: [pskv.prefill_attn_paged(d.layout, qp, pcu_dev, pcu, d.tables, d.lens, d.case.seq_lens, scale, stream=s)],
        "merge_partials": lambda s: [pskv.merge_partials(m, l, o, stream=s)],
    }


@pytest.fixture(scope="module")
def table():
    return calls()


NAMES = ["decode_attn_latent", "decode_attn_latent, Python", "decode_attn_latent, one piece", "prefill_attn_expanded",
         "prefill_attn_expanded, Python", "verify_drafts", "decode_attn_splitkv", "decode_attn_multirow",
         "prefill_attn_paged", "merge_partials"]
SIZES = [1 << k for k in range(9, 27)]


@pytest.mark.parametrize("as_number", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_given_out_again_is_not_the_call_s(table, name, as_number):
    """The current stream takes and fills memory of every size while the call waits on its stream."""
    want = table[name](None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(PAUSE)
    got = table[name](side.cuda_stream if as_number else side)
    taken = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(bool((t == 0x5A).all()) for t in taken)


@pytest.mark.parametrize("name", NAMES)
def test_memory_still_in_use_is_not_the_call_s(table, name):
    """Memory freed on the current stream, whose work on it still waits there, is not written by the call."""
    want = table[name](None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(3)]
    torch.cuda._sleep(PAUSE)
    for t in late:
        t.fill_(0x5A)
    del late, t
    got = table[name](side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_the_default_stream_by_number(table):
    for name in NAMES:
        want = table[name](None)
        got = table[name](0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
