"""Sizes that the decode calls refuse (no GPU needed: the fake device pointers are never dereferenced)."""

import ctypes

import pytest

from sparse_mla_attention_gb300 import _lib
from sparse_mla_attention_gb300._lib import SmlaPagedDims
from test_decode_api import _addrs, _weights, lib  # noqa: F401 (a fixture)


@pytest.mark.parametrize("T,H,fine", [(1 << 21, 16, True), (1 << 18, 128, True), ((1 << 21) + 1, 16, False),
                                      ((1 << 18) + 1, 128, False), (1 << 24, 128, False)])
def test_weights_refuse_more_rows_of_q_than_a_wait_covers(lib, T, H, fine):  # noqa: F811
    # (the sequences of a call may have any share of its tokens: one with all of them is the longest pass)
    size = ctypes.c_size_t(0)
    dims = SmlaPagedDims(T=T, H=H, D=512, topk=0, B=4, max_pages=10, scale=0.0)
    assert lib.smla_weights_workspace_size(dims, ctypes.byref(size)) == (_lib.SMLA_OK if fine else _lib.SMLA_ERR_SHAPE)
    # so many tokens' tensors do not fit between the fake addresses; a call within the limit gets past the sizes
    code = _weights(lib, _addrs(), T=T, H=H)
    assert (code != _lib.SMLA_ERR_SHAPE) if fine else (code == _lib.SMLA_ERR_SHAPE)
