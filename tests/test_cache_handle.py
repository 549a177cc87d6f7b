"""The cache's handle names its tensors to the library once: others cannot be put in their place."""

import pytest
import torch

import sparse_mla_attention_gb300 as smla


@pytest.mark.parametrize("name", ["pages", "scales", "refcount"])
def test_tensors_of_a_handle_cannot_be_replaced(name):
    handle = object.__new__(smla.PagedCache)          # (a whole one needs CUDA tensors)
    with pytest.raises(AttributeError):
        setattr(handle, name, torch.zeros(4, dtype=torch.int32))


@pytest.mark.gpu
def test_counts_are_copied_into_the_handle():
    cache = smla.PagedCache.empty(8, 16, 16)
    table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    cache.refcount[:3] = 1                            # three pages of somebody else
    smla.cache_alloc(cache, table, torch.tensor([20], dtype=torch.int32, device="cuda"))
    assert table.tolist() == [[3, 4]]
    smla.cache_free(cache, table)
    new, count = smla.cache_compact(cache, table)
    with pytest.raises(AttributeError):
        cache.refcount = count.zero_()
    cache.refcount.copy_(count)
    smla.cache_alloc(cache, table, torch.tensor([20], dtype=torch.int32, device="cuda"))
    assert table.tolist() == [[0, 1]]
