"""A workspace whose buffer a captured graph holds."""

import weakref

import pytest
import torch

import sparse_mla_attention_gb300 as smla
from sparse_mla_attention_gb300 import api


def test_buffers_that_a_capture_used_are_kept(monkeypatch):
    # (on the CPU, with the capture played by a flag)
    state = {"capturing": False}
    monkeypatch.setattr(api, "_capturing", lambda buf: state["capturing"], raising=False)
    ws = smla.Workspace("cpu")
    eager = weakref.ref(ws.get(1000))
    assert ws.get(2000).numel() == 2000
    assert eager() is None                                  # nobody holds its address
    state["capturing"] = True
    first = weakref.ref(ws.get(1500))
    assert first().numel() == 2000
    state["capturing"] = False
    assert ws.get(4000).numel() == 4000 and first() is not None
    third = weakref.ref(ws.get(3000))
    assert ws.get(8000).numel() == 8000 and third() is None and first() is not None
    state["capturing"] = True
    grown_in_capture = weakref.ref(ws.get(16000))
    state["capturing"] = False
    ws.get(32000)
    assert grown_in_capture() is not None and first() is not None
    del ws
    assert first() is None and grown_in_capture() is None


@pytest.mark.gpu
def test_a_replay_after_the_workspace_grew_touches_nothing_else():
    # a graph of an allocation is captured on a small workspace; a larger call makes the workspace grow; tensors
    # made afterwards must not lie where the graph's calls write, and its result must stay right
    cache = smla.PagedCache.empty(64, 16, 16)
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 0, 64], dtype=torch.int32, device="cuda")
    ws = smla.Workspace("cuda")
    smla.cache_alloc(cache, table, lens, workspace=ws)
    want = table.clone()
    size = ws.buf.numel()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smla.cache_alloc(cache, table, lens, workspace=ws, check_status=False)
    ws.get(64 << 20)
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(2):
        table.fill_(-1)
        cache.refcount.zero_()
        graph.replay()
        assert torch.equal(table, want)
    assert all(bool((t == 7).all()) for t in others)
