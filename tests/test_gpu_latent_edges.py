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
