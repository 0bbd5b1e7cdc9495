"""The CTA pairs of the latent kernels over long runs of tiles: whatever one CTA hands to the
other has to be there every time, so repeated calls agree bit for bit and with f64."""
import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from latent_cases import LatentCase, check_attention, normal
from test_gpu_latent import expanded_reference, vmax

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,dc,heads,tokens,page", [
    ([20003, 9001], 512, 128, 1, 256), ([12077, 130, 64], 256, 100, 3, 16), ([30001], 512, 32, 5, 48)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_repeats(lens, dc, heads, tokens, page, dtype):
    c = LatentCase(21, lens, dc, page, heads, tokens)
    ws = pskv.latent_workspace(c.layout, c.lens_host, tokens, heads, table_stride=c.table.shape[1])
    out = c.run(workspace=ws, out_dtype=dtype)
    check_attention(out, c.reference(), vmax(c))
    for splits in (0, 1):
        want = c.run(num_splits=splits, workspace=ws, out_dtype=dtype)
        check_attention(want, c.reference(), vmax(c))
        got = [c.run(num_splits=splits, workspace=ws, out_dtype=dtype) for _ in range(20)]
        assert all(torch.equal(want, o) for o in got)
    assert int(c.status[0]) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_expanded_repeats(dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(22)
    new, old = [1500, 3, 700, 129], [0, 2000, 77, 1]
    cq = [0] + np.cumsum(new).tolist()
    ck = [0] + np.cumsum([a + b for a, b in zip(new, old)]).tolist()
    q, kv, rot = normal(gen, cq[-1], 24, 192), normal(gen, ck[-1], 24, 256), normal(gen, ck[-1], 64)
    cu = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (cq, ck)]
    call = lambda: pskv.prefill_attn_expanded(q, kv, rot, cu[0], cq, cu[1], ck, 192 ** -0.5, out_dtype=dtype)
    out = call()
    check_attention(out, expanded_reference(q, kv, rot, cq, ck, 192 ** -0.5), float(kv.abs().max()))
    got = [call() for _ in range(20)]
    assert all(torch.equal(out, o) for o in got)
