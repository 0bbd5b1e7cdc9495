"""A latent scratch tensor sized once serves shorter and smaller batches, which may need more than the
longest lengths' own plan."""
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import LatentCase, check_attention
from test_gpu_latent import vmax

pytestmark = pytest.mark.gpu


def test_one_scratch_for_shorter_batches():
    heads, longest, rows = 32, 1500, 40
    first = LatentCase(41, [longest] * rows, heads=heads)
    need = lambda c: pskv.decode_attn_latent_workspace_bytes(c.layout, c.lens_host, c.table.shape[1], c.tokens, heads)
    ws = pskv.latent_workspace(first.layout, first.lens_host, 3, heads, bound=True)
    ws.fill_(0xFF)
    assert need(first) == 0 and pskv.latent_workspace(first.layout, first.lens_host, 1, heads) is None
    more = False
    for seed, lens, tokens in ((41, [longest] * rows, 1), (42, [longest] + [100] * (rows - 1), 1), (43, [1400], 3),
                               (44, [900, 1500, 7], 2), (45, [640] * 20, 3), (46, [1] * rows, 1)):
        c = LatentCase(seed, lens, heads=heads, tokens=tokens)
        more |= need(c) > need(first)
        assert need(c) <= ws.numel()
        check_attention(c.run(workspace=ws), c.reference(), vmax(c))
        assert int(c.status[0]) == 0
    assert more


@pytest.mark.parametrize("heads,tokens,longest,rows", [(128, 1, 40002, 8), (16, 5, 20001, 64), (100, 64, 3000, 3)])
def test_the_bound_covers_what_plans_need(heads, tokens, longest, rows):
    c = LatentCase(47, [200], heads=heads)
    bound = pskv.decode_attn_latent_workspace_bound(c.layout, longest, rows, tokens, heads)
    gen = torch.Generator().manual_seed(1)
    for _ in range(300):
        n, t = int(torch.randint(1, rows + 1, (1,), generator=gen)), int(torch.randint(1, tokens + 1, (1,), generator=gen))
        lens = (torch.rand(n, generator=gen) ** 3 * (longest - t)).int() + t
        need = pskv.decode_attn_latent_workspace_bytes(c.layout, lens.tolist(), -(-longest // 64), t, heads)
        assert need <= bound
