"""verify_drafts on the GPU against its definition in whole numbers."""
import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import verify_reference

pytestmark = pytest.mark.gpu


def inputs(seed, batch, t, vocab, dtype, guess, temperature=1.0, near=0.5):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    logits = torch.randn(batch, t + 1, vocab, generator=gen, device="cuda") * 2 / temperature
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :t] + near * torch.randn(batch, t, vocab, generator=gen, device="cuda"), -1)
    drafts = torch.zeros(batch, t, dtype=torch.int32, device="cuda") if t == 0 else \
        torch.multinomial(draft.reshape(-1, vocab), 1, generator=gen).reshape(batch, t).to(torch.int32)
    u = torch.rand(batch, t + 1, generator=gen, device="cuda")
    return target.to(dtype), None if guess else draft.to(dtype), drafts, u


def check(target, draft, drafts, u, num=None, **kw):
    tokens, accepted = pskv.verify_drafts(target, draft, drafts, u, num_drafts=num, **kw)
    want, many = verify_reference(target, draft, drafts, u, None if num is None else num.tolist())
    assert np.array_equal(accepted.cpu().numpy(), many)
    assert np.array_equal(tokens.cpu().numpy(), want)
    return many


@pytest.mark.parametrize("batch,t,vocab", [(1, 1, 1), (3, 2, 7), (2, 0, 500), (5, 4, 1000), (2, 33, 257),
                                           (1, 64, 65), (2, 3, 8192), (3, 1, 4099), (1, 2, 20001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("guess", [False, True])
def test_matches_the_definition(batch, t, vocab, dtype, guess):
    check(*inputs(batch * 1000 + vocab, batch, t, vocab, dtype, guess))


def test_ragged_counts_and_all_standing():
    target, draft, drafts, u = inputs(1, 6, 5, 900, torch.float32, False, near=0.0)
    num = torch.tensor([0, 1, 5, 3, 5, 2], dtype=torch.int32, device="cuda")
    many = check(target, draft, drafts, u, num)
    assert many.tolist() == num.tolist()  # p = q: every draft stands


def test_the_ends_of_u():
    """u at 0, just below 1, and outside [0, 1): the first and the last token with weight."""
    target, draft, drafts, u = inputs(2, 6, 1, 300, torch.float32, False)
    target[:, :, 0] = 0
    target[:, :, 299] = 0
    for k, v in enumerate((0.0, 1 - 2.0 ** -24, 1.0, -3.0, float("nan"), 2.0 ** -149)):
        u[k, :] = v
    check(target, draft, drafts, u)


def test_values_that_are_no_probabilities():
    target, draft, drafts, u = inputs(3, 4, 2, 400, torch.float32, False)
    target[0, 0, 5], target[1, 1, 7], target[2, :, :50] = float("nan"), -0.25, float("inf")
    draft[3, 0, :] = float("nan")
    draft[0, 1, 9] = -float("inf")
    check(target, draft, drafts, u)


def test_nothing_left_of_the_target():
    """p below q everywhere: the draw is from p; no weight at all: -1 and a fault bit."""
    target, draft, drafts, u = inputs(4, 3, 2, 333, torch.float32, False)
    draft = target[:, :2] * 1.5
    u[:, :2] = 0.999
    target[2] = 0
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    many = check(target, draft.contiguous(), drafts, u, status=status)
    assert many.tolist() == [0, 0, 0] and int(status[0]) == pskv.PSKV_FAULT_EMPTY_ROW


def test_bad_drafts_and_counts_are_flagged():
    target, draft, drafts, u = inputs(5, 3, 3, 100, torch.float32, False, near=0.0)
    drafts[0, 1], drafts[1, 0] = 100, -1
    for d in (draft, None):
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        many = check(target, d, drafts, u, status=status)
        assert many[1] == 0 and int(status[0]) == pskv.PSKV_FAULT_BAD_TOKEN
    drafts.clamp_(0, 99)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    check(target, draft, drafts, u, torch.tensor([-2, 9, 3], dtype=torch.int32, device="cuda"), status=status)
    assert int(status[0]) == pskv.PSKV_FAULT_BAD_LENGTH


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_off_16_bytes(dtype):
    """Tables that begin between 16-byte boundaries, and rows of a length that does not keep one."""
    target, draft, drafts, u = inputs(6, 2, 2, 1003, dtype, False)
    a = torch.empty(target.numel() + 1, dtype=dtype, device="cuda")[1:].view(target.shape).copy_(target)
    b = torch.empty(draft.numel() + 3, dtype=dtype, device="cuda")[3:].view(draft.shape).copy_(draft)
    check(a, b, drafts, u)


def test_large_vocabulary_and_wide_ranges():
    """Weights over many powers of two (down to 2^-60): whole-number sums, one answer."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    e = -60 * torch.rand(2, 2, 131072, generator=gen, device="cuda")
    target = torch.exp2(e)
    target /= target.sum(-1, keepdim=True)
    drafts = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for k in range(4):
        u = torch.rand(2, 2, generator=gen, device="cuda")
        check(target, None, drafts, u)


def test_capture_and_streams():
    target, draft, drafts, u = inputs(8, 4, 3, 5000, torch.float32, False)
    tokens = torch.empty(4, 4, dtype=torch.int32, device="cuda")
    accepted = torch.empty(4, dtype=torch.int32, device="cuda")
    pskv.verify_drafts(target, draft, drafts, u, tokens=tokens, accepted=accepted)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pskv.verify_drafts(target, draft, drafts, u, tokens=tokens, accepted=accepted)
    for k in range(3):
        u.copy_(torch.rand(u.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(k)))
        graph.replay()
        want, many = verify_reference(target, draft, drafts, u)
        assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(accepted.cpu().numpy(), many)


def test_python_refusals():
    target, draft, drafts, u = inputs(9, 2, 2, 50, torch.float32, False)
    with pytest.raises(ValueError):
        pskv.verify_drafts(target, draft[:, :1].contiguous(), drafts, u)
    with pytest.raises(TypeError):
        pskv.verify_drafts(target, draft.to(torch.bfloat16), drafts, u)
    with pytest.raises(TypeError):
        pskv.verify_drafts(target.half(), None, drafts, u)
    with pytest.raises(ValueError):
        pskv.verify_drafts(target, draft, drafts, u[:, :2].contiguous())
    with pytest.raises(TypeError):
        pskv.verify_drafts(target, draft, drafts.long(), u)
