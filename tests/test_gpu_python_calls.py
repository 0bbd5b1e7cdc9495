"""The latent operators without their compiled calls give the same results and the same refusals."""
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import LatentCase, normal
from paged_split_kv_attn_gb300 import _binding as B

pytestmark = pytest.mark.gpu


def results():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(51)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    c = LatentCase(51, [700, 65, 0], heads=24, tokens=2)
    out = [c.run(), c.run(num_splits=1, out_dtype=torch.float32), c.run(num_splits=3)]
    q, kv, rot = normal(gen, 90, 2, 192), normal(gen, 120, 2, 256), normal(gen, 120, 64)
    cu = dev([0, 30, 90]), dev([0, 50, 120])
    out.append(pskv.prefill_attn_expanded(q, kv, rot, cu[0], [0, 30, 90], cu[1], [0, 50, 120], 0.1))
    target = torch.softmax(torch.randn(5, 3, 901, generator=gen, device="cuda"), -1)
    drafts, u = torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.rand(5, 3, generator=gen, device="cuda")
    out += pskv.verify_drafts(target, None, drafts, u)
    pool = torch.zeros(4, 1, 64, 576, dtype=torch.bfloat16, device="cuda")
    layout, ang = pskv.paged_kv_layout_create(pool, None), torch.rand(800, 32, generator=gen, device="cuda")
    turned = torch.empty(2, 5, 64, dtype=torch.bfloat16, device="cuda")
    pskv.kv_prep_append_latent(layout, normal(gen, 2, 576), dev([0, 1]), dev([70, 3]), dev([[0, 1], [2, 3]]), dev([2, 2]),
                               1e-6, None, ang, ang, q=normal(gen, 2, 5, 64), q_out=turned)
    with pytest.raises(pskv.PskvError):
        pskv.decode_attn_latent(c.layout, c.q, c.table, c.lens, [700, 65, 1], c.scale)
    return out + [pool, turned]


def test_python_forms_alone(monkeypatch):
    want = results()
    assert B._calls is not None and B._calls is not B._PythonCalls, "the compiled calls were not built"
    monkeypatch.setattr(B, "_calls", B._PythonCalls)
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
