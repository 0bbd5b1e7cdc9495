"""A search of sample_tokens that does not end in the passes it may take is reported, and its row counts as empty: in a
library built with a bound that rows do reach."""
import ctypes

import numpy as np
import pytest
import torch

import paged_split_kv_attn_gb300 as pskv
from paged_split_kv_attn_gb300 import _binding as B
from paged_split_kv_attn_gb300 import build as pskv_build
from tree_cases import sample_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=[1, 2])
def bounded(request, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("lib") / "libpskv_bounded.so")
    pskv_build.build(out=out, defines={"PSKV_SAMPLE_PASSES": request.param})
    lib = ctypes.CDLL(out)
    P, I = ctypes.c_void_p, ctypes.c_int32
    lib.sample_tokens.argtypes = [P, I, ctypes.c_int64, I, I, I, ctypes.POINTER(B.SampleDesc), P, P, P, I, P, P]
    lib.passes = request.param
    return lib


@pytest.mark.parametrize("rows,vocab", [(12, 30000), (200, 5000)])  # pieces in shared memory, and several CTAs an SM
@pytest.mark.parametrize("some,part", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("drawn,shown", [(True, True), (True, False), (False, True)])
def test_rows_past_the_bound_are_empty(bounded, rows, vocab, some, part, drawn, shown):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    l = torch.randn(rows, vocab, generator=gen, device="cuda") * 2.5
    l[::3] *= 1e-4       # nearly equal weights: finer levels
    l[1::3, ::2] = -40.0
    u = torch.rand(rows, generator=gen, device="cuda")
    k = torch.full((rows,), vocab // 3, dtype=torch.int32, device="cuda")
    k[5::7] = 20
    p = torch.full((rows,), 0.9, device="cuda")
    tokens = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    probs, status = torch.full((rows, vocab), 7.0, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    f = B.SampleDesc(None, k.data_ptr() if some else None, p.data_ptr() if part else None, None)
    rc = bounded.sample_tokens(l.data_ptr(), 0, vocab, rows, 1, vocab, ctypes.byref(f), u.data_ptr() if drawn else None,
                               tokens.data_ptr() if drawn else None, probs.data_ptr() if shown else None, 0, status.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    kw = dict(**({"top_k": k.tolist()} if some else {}), **({"top_p": p.tolist()} if part else {}))
    want, dist = sample_reference(l[:, None], u[:, None], **kw)
    gone = (tokens == -1).cpu().numpy() if drawn else (probs == 0).all(1).cpu().numpy()
    assert int(status[0]) == (pskv.PSKV_FAULT_BAD_STATE if gone.any() else 0)
    assert gone.any() or bounded.passes > 1  # (nearly equal weights take two passes at least)
    if drawn:
        assert np.array_equal(tokens.cpu().numpy()[~gone], want[~gone, 0])
    if shown:
        got = probs.double().cpu().numpy()
        assert (got[gone] == 0).all() and (np.abs(got - dist[:, 0])[~gone] <= 2.0 ** -23 * dist[~gone, 0]).all()
    # the library itself searches on
    assert np.array_equal(pskv.sample_tokens(l, u, **{n: t for n, t in (("top_k", k), ("top_p", p)) if n in kw}).cpu().numpy(), want[:, 0])
