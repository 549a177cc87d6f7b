"""Host-side validation of the paged-cache entry points (no GPU needed): bad
arguments return their error code before any CUDA call, so the fake device
pointers below are never dereferenced."""

import ctypes

import pytest
import torch

import sparse_mla_attention_gb300 as smla
from sparse_mla_attention_gb300 import _lib, build as smla_build
from sparse_mla_attention_gb300._lib import SmlaCache, SmlaPagedDims

GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return _lib.load()


def _at(i, off=0):
    return ctypes.c_void_p((i + 1) * GB + off)


NAMES = ["pages", "scales", "refcount", "table", "lens", "q", "seq", "topk", "sink", "o", "lse", "ws",
         "start", "cu", "rows", "parents", "child", "src", "dst", "nt", "nr"]


def _addrs(**over):
    a = {k: _at(i) for i, k in enumerate(NAMES)}
    a.update(over)
    return a


def _cache(a, **over):
    kw = dict(num_pages=100, page_size=64, scale_block=32, D=512)
    kw.update(over)
    return SmlaCache(pages=a["pages"].value if a["pages"] else None,
                     scales=a["scales"].value if a["scales"] else None,
                     refcount=a["refcount"].value if a["refcount"] else None, **kw)


BIG = 1 << 29


def _attend(lib, a, cache=None, ws_bytes=BIG, **over):
    kw = dict(T=4, H=16, D=512, topk=8, B=4, max_pages=10, scale=0.0)
    kw.update(over)
    c = cache or _cache(a)
    return lib.smla_fwd_paged(a["q"], ctypes.byref(c), a["table"], a["seq"], a["lens"], a["topk"], a["sink"],
                              a["o"], a["lse"], ctypes.byref(SmlaPagedDims(**kw)), a["ws"], ws_bytes, None)


def _write(lib, a, cache=None, B=4, max_pages=10, n=7, ws_bytes=4096):
    c = cache or _cache(a)
    return lib.smla_cache_write(ctypes.byref(c), a["table"], a["start"], a["cu"], a["rows"], B, max_pages, n,
                                a["ws"], ws_bytes, None)


def _alloc(lib, a, cache=None, B=4, max_pages=10, ws_bytes=BIG):
    c = cache or _cache(a)
    return lib.smla_cache_alloc(ctypes.byref(c), a["table"], a["lens"], B, max_pages, a["ws"], ws_bytes, None)


def _fork(lib, a, cache=None, B=4, n=3, max_pages=10, ws_bytes=BIG):
    c = cache or _cache(a)
    return lib.smla_cache_fork(ctypes.byref(c), a["table"], a["lens"], a["parents"], a["child"], B, n, max_pages,
                               a["ws"], ws_bytes, None)


def _free(lib, a, cache=None, rows="start", B=4, n=4, max_pages=10, ws_bytes=BIG):
    c = cache or _cache(a)
    return lib.smla_cache_free(ctypes.byref(c), a["table"], a[rows] if rows else None, B, n, max_pages, a["ws"],
                               ws_bytes, None)


def _compact(lib, a, cache=None, B=4, max_pages=10, ws_bytes=BIG):
    c = cache or _cache(a)
    return lib.smla_cache_compact(ctypes.byref(c), a["table"], a["nt"], a["nr"], B, max_pages, a["ws"], ws_bytes,
                                  None)


def _copy(lib, a, cache=None, n=3, ws_bytes=BIG):
    c = cache or _cache(a)
    return lib.smla_cache_copy_pages(ctypes.byref(c), a["src"], a["dst"], n, a["ws"], ws_bytes, None)


CALLS = [_attend, _write, _alloc, _fork, _free, _compact, _copy]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("change", [dict(page_size=48), dict(page_size=8), dict(page_size=512),
                                    dict(scale_block=8), dict(scale_block=128, page_size=64), dict(num_pages=0),
                                    dict(num_pages=1 << 25, page_size=64)])
def test_unsupported_caches_are_refused(lib, call, change):
    a = _addrs()
    assert call(lib, a, cache=_cache(a, **change)) == _lib.SMLA_ERR_CACHE


@pytest.mark.parametrize("call", CALLS)
def test_common_pointer_rules(lib, call):
    a = _addrs()
    assert call(lib, a, cache=_cache(a, D=256)) == _lib.SMLA_ERR_D512
    a = _addrs(pages=None)
    assert call(lib, a) == _lib.SMLA_ERR_NULL
    a = _addrs(ws=None)
    assert call(lib, a) == _lib.SMLA_ERR_NULL
    a = _addrs(scales=_at(1, 4))
    assert call(lib, a) == _lib.SMLA_ERR_ALIGN
    assert call(lib, _addrs(), ws_bytes=16) == _lib.SMLA_ERR_WORKSPACE


@pytest.mark.parametrize("call", [_alloc, _fork, _free, _compact])
def test_page_calls_need_refcounts(lib, call):
    assert call(lib, _addrs(refcount=None)) == _lib.SMLA_ERR_NULL


@pytest.mark.parametrize("change,code", [
    (dict(D=128), _lib.SMLA_ERR_D512), (dict(H=24), _lib.SMLA_ERR_SHAPE), (dict(H=144), _lib.SMLA_ERR_SHAPE),
    (dict(H=0), _lib.SMLA_ERR_SHAPE), (dict(T=-1), _lib.SMLA_ERR_SHAPE), (dict(B=0), _lib.SMLA_ERR_SHAPE),
    (dict(max_pages=0), _lib.SMLA_ERR_SHAPE), (dict(max_pages=1 << 25), _lib.SMLA_ERR_SHAPE),
    (dict(topk=0), _lib.SMLA_ERR_ARG), (dict(topk=-1), _lib.SMLA_ERR_SHAPE),
    (dict(T=1 << 20, topk=1 << 12), _lib.SMLA_ERR_SHAPE),
    (dict(scale=float("inf")), _lib.SMLA_ERR_ARG), (dict(scale=-0.5), _lib.SMLA_ERR_ARG),
])
def test_attend_rejects_bad_dims(lib, change, code):
    assert _attend(lib, _addrs(), **change) == code


def test_attend_rejects_bad_pointers(lib):
    for name in ("q", "table", "lens", "o", "lse"):
        assert _attend(lib, _addrs(**{name: None})) == _lib.SMLA_ERR_NULL
    assert _attend(lib, _addrs(topk=None)) == _lib.SMLA_ERR_ARG
    assert _attend(lib, _addrs(seq=None), T=5) == _lib.SMLA_ERR_SHAPE      # a token without a row of its own
    a = _addrs(); a["o"] = a["q"]
    assert _attend(lib, a) == _lib.SMLA_ERR_OVERLAP
    a = _addrs(); a["lse"] = a["pages"]
    assert _attend(lib, a) == _lib.SMLA_ERR_OVERLAP
    a = _addrs(topk=_at(7, 8))
    assert _attend(lib, a) == _lib.SMLA_ERR_ALIGN


def test_write_rejections(lib):
    for name in ("table", "start", "cu", "rows"):
        assert _write(lib, _addrs(**{name: None})) == _lib.SMLA_ERR_NULL
    assert _write(lib, _addrs(), n=-1) == _lib.SMLA_ERR_SHAPE
    assert _write(lib, _addrs(), B=(1 << 24) + 1) == _lib.SMLA_ERR_SHAPE
    a = _addrs(); a["rows"] = a["pages"]
    assert _write(lib, a) == _lib.SMLA_ERR_OVERLAP


def test_page_call_rejections(lib):
    assert _alloc(lib, _addrs(table=None)) == _lib.SMLA_ERR_NULL
    assert _fork(lib, _addrs(parents=None)) == _lib.SMLA_ERR_NULL
    assert _fork(lib, _addrs(), n=-1) == _lib.SMLA_ERR_SHAPE
    a = _addrs(); a["child"] = a["table"]
    assert _fork(lib, a) == _lib.SMLA_ERR_OVERLAP
    assert _free(lib, _addrs(), rows=None, n=3) == _lib.SMLA_ERR_SHAPE     # all rows means B of them
    a = _addrs(); a["nt"] = a["table"]
    assert _compact(lib, a) == _lib.SMLA_ERR_OVERLAP
    a = _addrs(); a["nr"] = a["refcount"]
    assert _compact(lib, a) == _lib.SMLA_ERR_OVERLAP
    assert _copy(lib, _addrs(dst=None)) == _lib.SMLA_ERR_NULL
    assert _copy(lib, _addrs(), n=-2) == _lib.SMLA_ERR_SHAPE


@pytest.mark.parametrize("call", CALLS)
def test_valid_calls_reach_the_device_check(lib, call):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; valid calls are covered by the GPU tests")
    assert call(lib, _addrs()) in (_lib.SMLA_ERR_CUDA, _lib.SMLA_ERR_ARCH)


def test_status_strings(lib):
    for code in (_lib.SMLA_ERR_PAGES, _lib.SMLA_ERR_REFCOUNT, _lib.SMLA_ERR_CACHE):
        s = lib.smla_status_string(code)
        assert s and s != b"unknown status code"


def test_python_handle_refuses_what_it_cannot_hold():
    pages = torch.zeros((4, 64, 512), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales, count = torch.zeros(4, 2), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        smla.PagedCache(pages, scales, count)
    with pytest.raises(TypeError, match="pages"):
        smla.PagedCache(pages.view(torch.uint8), scales, count)
    with pytest.raises(ValueError, match="divide"):
        smla.PagedCache.empty(4, 64, 48, device="cpu")
    with pytest.raises(TypeError, match="q must be"):
        smla.sparse_mla_fwd_paged(torch.zeros(1, 16, 512), None, count, count)
