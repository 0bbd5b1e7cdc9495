"""verify_drafts with its clusters on their shortest way to one another's shared memory: no draft
and few tokens, far more rows than the GPU holds at a time, so that clusters start in the places
others leave."""
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import verify_reference

pytestmark = pytest.mark.gpu


def tables(seed, batch, t, vocab):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    target = torch.softmax(torch.randn(batch, t + 1, vocab, generator=gen, device="cuda"), -1)
    drafts = torch.randint(vocab, (batch, t), generator=gen, device="cuda").to(torch.int32)
    return target, drafts, torch.rand(batch, t + 1, generator=gen, device="cuda")


@pytest.mark.parametrize("t", [0, 1])
def test_many_rows_of_few_tokens(t):
    target, drafts, u = tables(11 + t, 1500, t, 9)
    want, many = verify_reference(target, None, drafts, u)
    want, many = torch.from_numpy(want).cuda(), torch.from_numpy(many).cuda()
    for _ in range(10):
        tokens, accepted = pskv.verify_drafts(target, None, drafts, u)
        assert torch.equal(tokens, want) and torch.equal(accepted, many)


def test_rows_that_try_twice():
    """Nothing left of the target (or nothing at all): the second try's stores follow the first's barrier."""
    target, drafts, u = tables(13, 1000, 1, 5)
    draft = (2 * target[:, :1]).contiguous()
    target[::2] = 0
    u[:, 0] = 1 - 2.0 ** -24
    want, many = verify_reference(target, draft, drafts, u)
    for _ in range(5):
        tokens, accepted = pskv.verify_drafts(target, draft, drafts, u)
        assert torch.equal(tokens, torch.from_numpy(want).cuda())
        assert torch.equal(accepted, torch.from_numpy(many).cuda())


def test_two_streams_at_once():
    cases = [tables(s, 700, 1, 300) for s in (14, 15)]
    want = [verify_reference(c[0], None, *c[1:]) for c in cases]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, c in zip(sides, cases):
            with torch.cuda.stream(s):
                got.append(pskv.verify_drafts(c[0], None, c[1], c[2]))
    torch.cuda.synchronize()
    for k, (tokens, accepted) in enumerate(got):
        assert torch.equal(tokens.cpu(), torch.from_numpy(want[k % 2][0]))
        assert torch.equal(accepted.cpu(), torch.from_numpy(want[k % 2][1]))
