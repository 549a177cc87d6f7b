"""Host-side validation of the decode loop's entry points (accumulated weights, eviction, reordering, beam selection; no
GPU needed): bad arguments return their error code before any CUDA call, so the fake device pointers below are never
dereferenced. And the 64-bit models' own rules for ties and odd values."""

import ctypes

import numpy as np
import pytest
import torch

import decode_reference as M
import sparse_mla_attention_gb300 as smla
from sparse_mla_attention_gb300 import _lib, build as smla_build
from sparse_mla_attention_gb300._lib import SmlaCache, SmlaPagedDims

GB = 1 << 30
BIG = 1 << 29


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return _lib.load()


NAMES = ["pages", "scales", "refcount", "table", "lens", "q", "cu", "lse", "earlier", "weights", "ws", "nt", "nl", "nw",
         "kept", "parents", "logits", "scores", "done", "tokens", "best"]


def _at(name, off=0):
    return ctypes.c_void_p((NAMES.index(name) + 1) * GB + off)


def _addrs(**over):
    a = {k: _at(k) for k in NAMES}
    a.update(over)
    return a


def _cache(a, **over):
    kw = dict(num_pages=100, page_size=64, scale_block=32, D=512)
    kw.update(over)
    v = lambda k: a[k].value if a[k] else None
    return SmlaCache(pages=v("pages"), scales=v("scales"), refcount=v("refcount"), **kw)


def _weights(lib, a, cache=None, ws_bytes=BIG, decay=0.5, **over):
    kw = dict(T=4, H=16, D=512, topk=0, B=4, max_pages=10, scale=0.0)
    kw.update(over)
    c = cache or _cache(a)
    return lib.smla_cache_weights(a["q"], ctypes.byref(c), a["table"], a["cu"], a["lens"], a["lse"], a["earlier"], decay,
                                  a["weights"], ctypes.byref(SmlaPagedDims(**kw)), a["ws"], ws_bytes, None)


def _evict(lib, a, cache=None, ws_bytes=BIG, B=4, max_pages=10, keep=100, first=3, recent=20):
    c = cache or _cache(a)
    return lib.smla_cache_evict(ctypes.byref(c), a["table"], a["lens"], a["weights"], a["nt"], a["nl"], a["nw"], a["kept"],
                                B, max_pages, keep, first, recent, a["ws"], ws_bytes, None)


def _reorder(lib, a, cache=None, ws_bytes=BIG, B=4, n=5, max_pages=10):
    c = cache or _cache(a)
    return lib.smla_cache_reorder(ctypes.byref(c), a["table"], a["lens"], a["parents"], a["weights"], a["nt"], a["nl"],
                                  a["nw"], B, n, max_pages, a["ws"], ws_bytes, None)


def _select(lib, a, ws_bytes=BIG, type=1, stride=1000, eos=3, B=2, K=4, V=1000, n=4):
    return lib.smla_beam_select(a["logits"], type, stride, a["scores"], a["done"], eos, a["parents"], a["tokens"], a["best"],
                                B, K, V, n, a["ws"], ws_bytes, None)


CACHE_CALLS = [_weights, _evict, _reorder]
CALLS = CACHE_CALLS + [_select]


@pytest.mark.parametrize("call", CACHE_CALLS)
@pytest.mark.parametrize("change", [dict(page_size=48), dict(page_size=512), dict(scale_block=8),
                                    dict(scale_block=128, page_size=64), dict(num_pages=0),
                                    dict(num_pages=1 << 25, page_size=64)])
def test_unsupported_caches_are_refused(lib, call, change):
    a = _addrs()
    assert call(lib, a, cache=_cache(a, **change)) == _lib.SMLA_ERR_CACHE


@pytest.mark.parametrize("call", CACHE_CALLS)
def test_common_pointer_rules(lib, call):
    a = _addrs()
    assert call(lib, a, cache=_cache(a, D=256)) == _lib.SMLA_ERR_D512
    for name in ("pages", "scales", "table", "lens", "ws"):
        assert call(lib, _addrs(**{name: None})) == _lib.SMLA_ERR_NULL
    assert call(lib, _addrs(table=_at("table", 4))) == _lib.SMLA_ERR_ALIGN
    assert call(lib, _addrs(weights=_at("weights", 4))) == _lib.SMLA_ERR_ALIGN
    assert call(lib, _addrs(), ws_bytes=16) == _lib.SMLA_ERR_WORKSPACE
    assert call(lib, _addrs(ws=_at("pages", 256))) == _lib.SMLA_ERR_OVERLAP
    for bad in (dict(B=-1), dict(B=(1 << 24) + 1), dict(max_pages=0), dict(max_pages=1 << 26)):
        assert call(lib, _addrs(), **bad) == _lib.SMLA_ERR_SHAPE


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), _lib.SMLA_ERR_SHAPE), (dict(H=8), _lib.SMLA_ERR_SHAPE), (dict(H=144), _lib.SMLA_ERR_SHAPE),
    (dict(H=40), _lib.SMLA_ERR_SHAPE), (dict(D=256), _lib.SMLA_ERR_D512), (dict(T=1 << 28), _lib.SMLA_ERR_SHAPE),
    (dict(topk=8), _lib.SMLA_ERR_ARG), (dict(scale=-1.0), _lib.SMLA_ERR_ARG), (dict(scale=float("inf")), _lib.SMLA_ERR_ARG),
    (dict(decay=float("nan")), _lib.SMLA_ERR_ARG), (dict(decay=float("inf")), _lib.SMLA_ERR_ARG)])
def test_weights_rejects_bad_dims(lib, change, code):
    assert _weights(lib, _addrs(), **change) == code


def test_weights_rejects_bad_pointers(lib):
    for name in ("q", "lse", "weights", "earlier"):
        assert _weights(lib, _addrs(**{name: None})) == _lib.SMLA_ERR_NULL
    assert _weights(lib, _addrs(cu=None), T=5) == _lib.SMLA_ERR_SHAPE
    # earlier may be weights itself, but not a part of it
    assert _weights(lib, _addrs(earlier=_at("weights", 256))) == _lib.SMLA_ERR_OVERLAP
    assert _weights(lib, _addrs(earlier=_at("weights"))) not in (_lib.SMLA_ERR_OVERLAP, _lib.SMLA_ERR_NULL)
    assert _weights(lib, _addrs(earlier=None), decay=0.0) != _lib.SMLA_ERR_NULL
    assert _weights(lib, _addrs(weights=_at("lse"))) == _lib.SMLA_ERR_OVERLAP
    size = ctypes.c_size_t(0)
    for bad in (dict(T=-1), dict(H=24), dict(B=-1)):
        kw = dict(T=4, H=16, D=512, topk=0, B=4, max_pages=10, scale=0.0)
        kw.update(bad)
        assert lib.smla_weights_workspace_size(SmlaPagedDims(**kw), ctypes.byref(size)) == _lib.SMLA_ERR_SHAPE


def test_evict_rejections(lib):
    for name in ("refcount", "weights", "nt", "nl", "nw", "kept"):
        assert _evict(lib, _addrs(**{name: None})) == _lib.SMLA_ERR_NULL
    for bad in (dict(keep=0), dict(keep=641)):
        assert _evict(lib, _addrs(), **bad) == _lib.SMLA_ERR_SHAPE
    for bad in (dict(first=-1), dict(recent=-1), dict(first=81, recent=20), dict(first=(1 << 31) - 1, recent=(1 << 31) - 1)):
        assert _evict(lib, _addrs(), **bad) == _lib.SMLA_ERR_ARG
    for out, src in (("nt", "table"), ("nl", "lens"), ("nw", "weights"), ("kept", "nt"), ("kept", "scales")):
        assert _evict(lib, _addrs(**{out: _at(src)})) == _lib.SMLA_ERR_OVERLAP
    size = ctypes.c_size_t(0)
    c = _cache(_addrs())
    for B, keep in ((-1, 5), (4, 0), ((1 << 24) + 1, 5)):
        assert lib.smla_cache_evict_workspace_size(ctypes.byref(c), B, keep, ctypes.byref(size)) == _lib.SMLA_ERR_SHAPE
    assert lib.smla_cache_evict_workspace_size(ctypes.byref(c), 4, 5, None) == _lib.SMLA_ERR_NULL


def test_reorder_rejections(lib):
    for name in ("refcount", "parents", "nt", "nl"):
        assert _reorder(lib, _addrs(**{name: None})) == _lib.SMLA_ERR_NULL
    assert _reorder(lib, _addrs(weights=None)) == _lib.SMLA_ERR_ARG
    assert _reorder(lib, _addrs(nw=None)) == _lib.SMLA_ERR_ARG
    for n in (-1, (1 << 24) + 1):
        assert _reorder(lib, _addrs(), n=n) == _lib.SMLA_ERR_SHAPE
    for out, src in (("nt", "table"), ("nl", "lens"), ("nw", "weights"), ("nl", "parents"), ("nt", "refcount")):
        assert _reorder(lib, _addrs(**{out: _at(src)})) == _lib.SMLA_ERR_OVERLAP
    size = ctypes.c_size_t(0)
    assert lib.smla_cache_reorder_workspace_size(-1, 3, ctypes.byref(size)) == _lib.SMLA_ERR_SHAPE


@pytest.mark.parametrize("change,code", [
    (dict(K=0), _lib.SMLA_ERR_SHAPE), (dict(K=65), _lib.SMLA_ERR_SHAPE), (dict(n=0), _lib.SMLA_ERR_SHAPE),
    (dict(n=65), _lib.SMLA_ERR_SHAPE), (dict(V=0), _lib.SMLA_ERR_SHAPE), (dict(V=(1 << 22) + 1), _lib.SMLA_ERR_SHAPE),
    (dict(B=-1), _lib.SMLA_ERR_SHAPE), (dict(B=1 << 24, K=64, V=1 << 22), _lib.SMLA_ERR_SHAPE),
    (dict(stride=-1), _lib.SMLA_ERR_SHAPE), (dict(stride=(1 << 63) - 1), _lib.SMLA_ERR_SHAPE), (dict(type=3), _lib.SMLA_ERR_ARG), (dict(type=-1), _lib.SMLA_ERR_ARG),
    (dict(eos=-1), _lib.SMLA_ERR_ARG), (dict(eos=1000), _lib.SMLA_ERR_ARG), (dict(ws_bytes=255), _lib.SMLA_ERR_WORKSPACE)])
def test_select_rejects_bad_sizes(lib, change, code):
    assert _select(lib, _addrs(), **change) == code


def test_select_rejects_bad_pointers(lib):
    for name in ("logits", "scores", "parents", "tokens", "best", "ws"):
        assert _select(lib, _addrs(**{name: None})) == _lib.SMLA_ERR_NULL
    assert _select(lib, _addrs(logits=_at("logits", 1))) == _lib.SMLA_ERR_ALIGN
    assert _select(lib, _addrs(logits=_at("logits", 2)), type=0) == _lib.SMLA_ERR_ALIGN
    assert _select(lib, _addrs(logits=_at("logits", 2))) != _lib.SMLA_ERR_ALIGN
    assert _select(lib, _addrs(scores=_at("scores", 2))) == _lib.SMLA_ERR_ALIGN
    for out, src in (("parents", "logits"), ("tokens", "scores"), ("best", "done"), ("ws", "logits"), ("tokens", "parents")):
        assert _select(lib, _addrs(**{out: _at(src)})) == _lib.SMLA_ERR_OVERLAP


@pytest.mark.parametrize("call", CALLS)
def test_valid_calls_reach_the_device_check(lib, call):
    if torch.cuda.is_available():
        pytest.skip("the fake pointers are for machines without a GPU")
    assert call(lib, _addrs()) == _lib.SMLA_ERR_CUDA


def test_python_calls_refuse_cpu_tensors():
    with pytest.raises(ValueError):
        smla.beam_select(torch.zeros(4, 10), torch.zeros(1, 4))
    with pytest.raises(TypeError):
        smla.beam_select(torch.zeros(4, 10), torch.zeros(1, 4, dtype=torch.float64))


# ------------------------------------------------------------------------------------------------ the models
def test_the_model_of_eviction_keeps_what_it_says():
    w = np.array([1.0, 5.0, 5.0, np.nan, -np.inf, 5.0, 0.0, 7.0, np.inf, 2.0])
    assert M.choose(w, 10, 10, 0, 0) == list(range(10))
    assert M.choose(w, 10, 3, 0, 0) == [1, 7, 8]       # of the fives the lowest
    assert M.choose(w, 10, 3, 1, 1) == [0, 8, 9]
    assert M.choose(w, 10, 9, 0, 0) == [0, 1, 2, 4, 5, 6, 7, 8, 9]      # NaN goes first
    assert M.choose(w, 10, 2, 1, 1) == [0, 9]
    assert M.choose(np.zeros(4), 4, 2, 0, 0) == [0, 1]


def test_the_model_of_selection():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.25, 0.25, 0.5]]))
    p, t, s = M.select(x, np.zeros((1, 2)), 4)
    assert p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[0, 2, 1, 2]]
    np.testing.assert_allclose(np.exp(s[0]), [0.5, 0.5, 0.25, 0.25])
    p, t, s = M.select(x, np.array([[-1.0, -np.inf]]), 5, done=np.array([[True, False]]), eos=1)
    assert p.tolist() == [[0, -1, -1, -1, -1]] and t[0, 0] == 1 and s[0, 0] == -1.0
    x[0, 1] = np.nan
    assert M.select(x, np.zeros((1, 2)), 2)[0].tolist() == [[1, 1]]
