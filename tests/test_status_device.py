"""A fault word on another device than the call's is refused before any launch (no GPU needed: the
tensors only say where they are)."""
import pytest
import torch

from paged_split_kv_attn_gb300 import _binding as B


class Elsewhere(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


def test_another_device():
    t = torch.zeros(4, dtype=torch.int32).as_subclass(Elsewhere)
    assert B._status(None, 0) is None
    assert B._status(t, 1) == t.data_ptr()
    with pytest.raises(ValueError):
        B._status(t, 0)
    with pytest.raises(TypeError):
        B._status(torch.zeros(4, dtype=torch.int64).as_subclass(Elsewhere), 1)


def test_layouts_ask_for_the_pool_s_device():
    pool = torch.zeros(2, 1, 64, 576, dtype=torch.bfloat16).as_subclass(Elsewhere)
    status = torch.zeros(4, dtype=torch.int32).as_subclass(Elsewhere)
    status.get_device = lambda: 0
    with pytest.raises(ValueError):
        B.paged_kv_layout_create(pool, None, status)
    with pytest.raises(ValueError):
        B.paged_kv_layout_create(pool[..., :512].contiguous(), pool[..., :512].contiguous(), status)
