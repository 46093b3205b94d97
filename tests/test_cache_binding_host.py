"""What the Python binding checks of a cache's tensors before any call, without a
GPU: CPU tensors stand in for CUDA ones, their device number set by the test."""
import pytest
import torch

import causal_gqa_attention_rmsnorm_gb300 as tb


@pytest.fixture
def on_gpu(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)


def rows(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_a_dense_lens_is_taken(on_gpu):
    lens = torch.tensor([3, 5, 7], dtype=torch.int32)
    c = tb.KVCache(rows(3, 2, 32, 64), rows(3, 2, 32, 64), lens).c()
    assert c.lens == lens.data_ptr() and (c.B, c.Hkv, c.T_max, c.dh) == (3, 2, 32, 64)


@pytest.mark.parametrize("paged", [False, True])
def test_a_lens_that_is_not_dense_is_refused(on_gpu, paged):
    """The kernels read and write B consecutive integers from its first one: a
    column of another tensor would lose its neighbours, an expanded entry what lies
    behind it."""
    bt = torch.zeros(3, 2, dtype=torch.int32) if paged else None
    shape = (8, 2, 16, 64) if paged else (3, 2, 32, 64)
    state = torch.zeros(3, 2, dtype=torch.int32)
    for lens in (state[:, 0], torch.zeros(6, dtype=torch.int32)[::2], torch.zeros(1, dtype=torch.int32).expand(3)):
        with pytest.raises(ValueError, match="lens"):
            tb.KVCache(rows(*shape), rows(*shape), lens, bt).c()
    # one sequence: every stride is dense
    one = tb.KVCache(rows(1, 2, 32, 64), rows(1, 2, 32, 64), state[:1, 1]).c()
    assert one.lens == state.data_ptr() + 4
