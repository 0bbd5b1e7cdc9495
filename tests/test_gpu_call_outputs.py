"""Outputs that a compiled call makes for itself come by torch.empty's way: deterministic mode fills them, dispatch
modes see them, as those of the Python forms."""
import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import paged_split_kv_attn_gb300 as pskv
from latent_cases import LatentCase, normal
from paged_split_kv_attn_gb300 import _binding as B
from tree_cases import Cache, i32, i64, random_masks

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["compiled", "Python"])
def form(request, monkeypatch):
    if request.param == "Python":
        monkeypatch.setattr(B, "_calls", B._PythonCalls)
    else:
        B._bind_calls(pskv.load_library())
        assert B._calls is not B._PythonCalls, "the compiled calls were not built"


class Made(TorchDispatchMode):
    """Shapes and types of the new tensors that go through the dispatcher."""

    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in str(func):
            self.made.append((tuple(out.shape), out.dtype))
        return out


def calls():
    """name -> (call of new outputs, their shapes and types)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(61)
    c = LatentCase(61, [300, 40], 256, 64, 8, 4)
    ws = pskv.latent_workspace(c.layout, c.lens_host, 4, 8)
    masks = i64(random_masks(np.random.default_rng(61), 2, 4))
    target = torch.softmax(torch.randn(5, 3, 901, generator=gen, device="cuda"), -1)
    logits = torch.randn(2, 4, 700, generator=gen, device="cuda")
    u = torch.rand(2, 4, generator=gen, device="cuda")
    drafts = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    rows = Cache(61, "latent256", [90, 100])
    path, kept = i32([[0, 2, -1, -1]] * 2), i32([2, 1])
    q, kv, rot = normal(gen, 90, 2, 192), normal(gen, 120, 2, 256), normal(gen, 120, 64)
    cu_q, cu_k = i32([0, 30, 90]), i32([0, 50, 120])
    bf16, whole = torch.bfloat16, torch.int32
    return {
        "decode_attn_latent": (lambda: pskv.decode_attn_latent(c.layout, c.q, c.table, c.lens, c.lens_host, c.scale, workspace=ws),
                               [((2, 4, 8, 256), bf16)]),
        "decode_attn_latent_tree": (lambda: pskv.decode_attn_latent_tree(c.layout, c.q, c.table, c.lens, c.lens_host, masks, c.scale,
                                                                         workspace=ws), [((2, 4, 8, 256), bf16)]),
        "prefill_attn_expanded": (lambda: pskv.prefill_attn_expanded(q, kv, rot, cu_q, [0, 30, 90], cu_k, [0, 50, 120], 0.1),
                                  [((90, 2, 128), bf16)]),
        "verify_drafts": (lambda: pskv.verify_drafts(target, None, drafts.new_zeros(5, 2), u.new_full((5, 3), 0.5)),
                          [((5, 3), whole), ((5,), whole)]),
        "sample_tokens": (lambda: pskv.sample_tokens(logits, u), [((2, 4), whole)]),
        "verify_tree": (lambda: pskv.verify_tree(drafts, masks, drafts), [((2, 4), whole)] * 2 + [((2,), whole)]),
        "kv_keep_tokens": (lambda: pskv.kv_keep_tokens(rows.layouts, rows.dev_table, rows.dev_lens, path, kept), [((2,), whole)]),
    }


@pytest.mark.parametrize("name", ["decode_attn_latent", "decode_attn_latent_tree", "prefill_attn_expanded", "verify_drafts",
                                  "sample_tokens", "verify_tree", "kv_keep_tokens"])
def test_dispatch_modes_see_new_outputs(form, name):
    call, want = calls()[name]
    call()
    with Made() as mode:
        call()
    assert all(mode.made.count(w) >= want.count(w) for w in want), mode.made


def test_deterministic_mode_fills_what_a_call_leaves(form):
    """Rows behind the device's last sequence are left as they were: as new memory they hold what was there, or the fill."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(62)
    q, kv, rot = normal(gen, 90, 2, 192), normal(gen, 120, 2, 256), normal(gen, 120, 64)
    cu_q, cu_k = i32([0, 30, 60]), i32([0, 50, 120])
    call = lambda: pskv.prefill_attn_expanded(q, kv, rot, cu_q, [0, 30, 90], cu_k, [0, 50, 120], 0.1)
    want = call()[:60].clone()
    torch.use_deterministic_algorithms(True)
    try:
        old = torch.full((90, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        del old  # (its memory is the next one's of this size)
        out = call()
    finally:
        torch.use_deterministic_algorithms(False)
    assert torch.equal(out[:60], want) and bool(out[60:].isnan().all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_distribution_alone_is_a_compiled_call(monkeypatch, dtype):
    """Without uniform numbers sample_tokens makes only probabilities: by the compiled call, to the Python form's bits."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(63)
    l = torch.randn(3, 2, 900, generator=gen, device="cuda").to(dtype)
    kw = dict(top_k=i32([5, 0, 900]), top_p=torch.tensor([0.5, 0.9, 1.0], device="cuda"))
    want, got = (torch.empty(3, 2, 900, dtype=dtype, device="cuda") for _ in range(2))
    with monkeypatch.context() as m:
        m.setattr(B, "_calls", B._PythonCalls)
        assert pskv.sample_tokens(l, None, probs=want, **kw) is None
    assert B._bind_calls(pskv.load_library()) is not B._PythonCalls, "the compiled calls were not built"
    with pytest.raises(pskv.PskvError):
        pskv.sample_tokens(l, None, **kw)
    with pytest.raises(pskv.PskvError):
        pskv.sample_tokens(l, None, tokens=torch.zeros(3, 2, dtype=torch.int32, device="cuda"), probs=got)
    monkeypatch.setattr(B, "_LIB", object())  # (what the Python form calls)
    assert pskv.sample_tokens(l, None, probs=got, **kw) is None
    torch.cuda.synchronize()
    assert torch.equal(got, want)
