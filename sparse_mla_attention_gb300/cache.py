"""Serving from a paged 8-bit cache: torch-facing wrappers (marshalling only).

``PagedCache`` is a handle on the pool (pages of e4m3 rows, a scale for each
block of rows, a reference count for each page). Block tables and lengths are
plain int32 tensors of the caller. Everything runs on the device, on the
current stream; no call reads a length or a table back. With
``check_status`` a call waits for the stream and raises if a kernel met a bad
index or too few free pages; without it the call only enqueues work and can
be captured into a CUDA graph.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import SmlaCache, SmlaPagedDims
from .api import D_HEAD, Workspace, _need, _ptr, _stream, device_status


class PagedCache:
    """A pool of pages for the kv rows of many sequences.

    pages    [num_pages, page_size, 512] float8_e4m3fn
    scales   [num_pages, page_size // scale_block] float32: row value = code * scale
    refcount [num_pages] int32: table entries that hold the page (0: free)

    page_size is 16, 32, 64, 128 or 256, scale_block 16, 32 or 64. The tensors
    are the caller's: the handle keeps them and the C struct that names them.
    """

    def __init__(self, pages: torch.Tensor, scales: torch.Tensor, refcount: torch.Tensor):
        _need(pages, "pages", torch.float8_e4m3fn, 3)
        _need(scales, "scales", torch.float32, 2)
        _need(refcount, "refcount", torch.int32, 1)
        n, ps, d = pages.shape
        if scales.shape[0] != n or refcount.shape[0] != n:
            raise ValueError("scales and refcount must have one row per page")
        if scales.shape[1] < 1 or ps % scales.shape[1] != 0:
            raise ValueError("scales must have page_size / scale_block columns")
        for name, t in (("scales", scales), ("refcount", refcount)):
            if t.device != pages.device:
                raise ValueError(f"{name} must be on {pages.device}, got {t.device}")
        self.pages, self.scales, self.refcount = pages, scales, refcount
        self.num_pages, self.page_size = n, ps
        self.scale_block = ps // scales.shape[1]
        self.device = pages.device
        self._c = SmlaCache(pages=pages.data_ptr(), scales=scales.data_ptr(),
                            refcount=refcount.data_ptr(), num_pages=n, page_size=ps,
                            scale_block=self.scale_block, D=d)
        self._ref = ctypes.byref(self._c)
        size = ctypes.c_size_t(0)
        _lib.check(_lib.load().smla_cache_workspace_size(self._ref, 0, ctypes.byref(size)), "PagedCache")

    @classmethod
    def empty(cls, num_pages: int, page_size: int = 64, scale_block: int = 64, device=None) -> "PagedCache":
        """A pool of free pages (their rows are whatever the memory held)."""
        dev = torch.device(device or "cuda")
        if scale_block < 1 or page_size % scale_block != 0:
            raise ValueError("scale_block must divide page_size")
        return cls(torch.empty((num_pages, page_size, D_HEAD), dtype=torch.float8_e4m3fn, device=dev),
                   torch.zeros((num_pages, page_size // scale_block), dtype=torch.float32, device=dev),
                   torch.zeros(num_pages, dtype=torch.int32, device=dev))

    def _workspace(self, workspace: Optional[Workspace], n: int) -> torch.Tensor:
        size = ctypes.c_size_t(0)
        _lib.check(_lib.load().smla_cache_workspace_size(self._ref, n, ctypes.byref(size)),
                   "smla_cache_workspace_size")
        return (workspace or Workspace(self.device)).get(size.value)


def _same_device(cache: PagedCache, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != cache.device:
            raise ValueError(f"{name} must be on {cache.device}, got {t.device}")


def _finish(code: int, where: str, ws: torch.Tensor, check_status: bool) -> None:
    _lib.check(code, where)
    if check_status:
        st = device_status(ws)
        if st != _lib.SMLA_OK:
            raise _lib.SmlaError(st, f"{where} (device)")


def sparse_mla_fwd_paged(q: torch.Tensor, cache: PagedCache, table: torch.Tensor, lens: torch.Tensor,
                         topk: Optional[torch.Tensor] = None, seq: Optional[torch.Tensor] = None,
                         sink: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                         workspace: Optional[Workspace] = None, check_status: bool = True,
                         out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
                         ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of query tokens over the cache: (o [T,H,512] bf16, lse [T,H] fp32).

    q [T,H,512] bf16; table [B, max_pages] int32; token t belongs to table row
    seq[t] (row t without ``seq``) and sees positions [0, lens[t]): all of
    them, or the picks topk[t, :] (positions, -1 masked). A token with lens 0
    (a padded slot) gets zeros. ``out`` = (o, lse) writes into the caller's
    tensors.
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(table, "table", torch.int32, 2)
    _need(lens, "lens", torch.int32, 1)
    T, H, D = q.shape
    if lens.shape[0] != T:
        raise ValueError("lens must have shape [T]")
    K = 0
    if topk is not None:
        _need(topk, "topk", torch.int32, 2)
        K = topk.shape[1]
        if topk.shape[0] != T or K < 1:
            raise ValueError("topk must have shape [T, K], K >= 1")
    if seq is not None:
        _need(seq, "seq", torch.int32, 1)
        if seq.shape[0] != T:
            raise ValueError("seq must have shape [T]")
    elif T > table.shape[0]:
        raise ValueError("without seq, table must have a row for each token")
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
        if sink.shape[0] != H:
            raise ValueError("sink must have shape [H]")
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
        _need(o, "o", torch.bfloat16, 3)
        _need(lse, "lse", torch.float32, 2)
        if o.shape != q.shape or tuple(lse.shape) != (T, H):
            raise ValueError("out must be (o [T,H,D], lse [T,H])")
    _same_device(cache, q=q, table=table, lens=lens, topk=topk, seq=seq, sink=sink, o=o, lse=lse)
    lib = _lib.load()
    dims = SmlaPagedDims(T, H, D, K, table.shape[0], table.shape[1], 0.0 if scale is None else float(scale))
    ref = ctypes.byref(dims)
    size = ctypes.c_size_t(0)
    _lib.check(lib.smla_paged_workspace_size(ref, ctypes.byref(size)), "smla_paged_workspace_size")
    ws = (workspace or Workspace(q.device)).get(size.value)
    _finish(lib.smla_fwd_paged(_ptr(q), cache._ref, _ptr(table), _ptr(seq), _ptr(lens), _ptr(topk),
                               _ptr(sink), _ptr(o), _ptr(lse), ref, _ptr(ws), ws.numel(),
                               _stream(q.device)),
            "smla_fwd_paged", ws, check_status)
    return o, lse


def cache_write(cache: PagedCache, table: torch.Tensor, start: torch.Tensor, cu_rows: torch.Tensor,
                rows: torch.Tensor, workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Write rows[cu_rows[b]:cu_rows[b+1]] (bf16 [n,512]) to the positions from start[b] on of
    the sequence in table row b, quantised block by block (smla_cache_write)."""
    _need(table, "table", torch.int32, 2)
    _need(start, "start", torch.int32, 1)
    _need(cu_rows, "cu_rows", torch.int32, 1)
    _need(rows, "rows", torch.bfloat16, 2)
    B = table.shape[0]
    if start.shape[0] != B or cu_rows.shape[0] != B + 1:
        raise ValueError("start must have shape [B] and cu_rows [B+1]")
    if rows.shape[1] != D_HEAD:
        raise ValueError("rows must have shape [n, 512]")
    _same_device(cache, table=table, start=start, cu_rows=cu_rows, rows=rows)
    ws = (workspace or Workspace(cache.device)).get(256)
    _finish(_lib.load().smla_cache_write(cache._ref, _ptr(table), _ptr(start), _ptr(cu_rows), _ptr(rows),
                                         B, table.shape[1], rows.shape[0], _ptr(ws), ws.numel(),
                                         _stream(cache.device)),
            "smla_cache_write", ws, check_status)


def cache_alloc(cache: PagedCache, table: torch.Tensor, lens: torch.Tensor,
                workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Give every sequence the pages that lens[b] rows need, in place on table and
    cache.refcount; lowest free pages first, all or nothing (smla_cache_alloc)."""
    _need(table, "table", torch.int32, 2)
    _need(lens, "lens", torch.int32, 1)
    B = table.shape[0]
    if lens.shape[0] != B:
        raise ValueError("lens must have shape [B]")
    _same_device(cache, table=table, lens=lens)
    ws = cache._workspace(workspace, B)
    _finish(_lib.load().smla_cache_alloc(cache._ref, _ptr(table), _ptr(lens), B, table.shape[1], _ptr(ws),
                                         ws.numel(), _stream(cache.device)),
            "smla_cache_alloc", ws, check_status)


def cache_fork(cache: PagedCache, table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
               out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
               check_status: bool = True) -> torch.Tensor:
    """Fork sequences: the table rows [n, max_pages] of the children of rows parents[i].

    Full pages are shared (refcount + 1), a partly filled last page is copied
    to a free one. All or nothing. ``out`` takes the child rows."""
    _need(table, "table", torch.int32, 2)
    _need(lens, "lens", torch.int32, 1)
    _need(parents, "parents", torch.int32, 1)
    B, max_pages = table.shape
    n = parents.shape[0]
    if lens.shape[0] != B:
        raise ValueError("lens must have shape [B]")
    child = torch.empty((n, max_pages), dtype=torch.int32, device=table.device) if out is None else out
    _need(child, "out", torch.int32, 2)
    if tuple(child.shape) != (n, max_pages):
        raise ValueError("out must have shape [n, max_pages]")
    _same_device(cache, table=table, lens=lens, parents=parents, out=child)
    ws = cache._workspace(workspace, n)
    _finish(_lib.load().smla_cache_fork(cache._ref, _ptr(table), _ptr(lens), _ptr(parents), _ptr(child), B, n,
                                        max_pages, _ptr(ws), ws.numel(), _stream(cache.device)),
            "smla_cache_fork", ws, check_status)
    return child


def cache_free(cache: PagedCache, table: torch.Tensor, rows: Optional[torch.Tensor] = None,
               workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Give back the pages of the table rows listed in ``rows`` (all rows without it): their
    entries become -1 and the pages' refcounts fall by one (smla_cache_free)."""
    _need(table, "table", torch.int32, 2)
    if rows is not None:
        _need(rows, "rows", torch.int32, 1)
    _same_device(cache, table=table, rows=rows)
    B = table.shape[0]
    n = B if rows is None else rows.shape[0]
    ws = (workspace or Workspace(cache.device)).get(256)
    _finish(_lib.load().smla_cache_free(cache._ref, _ptr(table), _ptr(rows), B, n, table.shape[1], _ptr(ws),
                                        ws.numel(), _stream(cache.device)),
            "smla_cache_free", ws, check_status)


def cache_compact(cache: PagedCache, table: torch.Tensor, workspace: Optional[Workspace] = None,
                  check_status: bool = True,
                  out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Move the last live pages into the holes before them: (new_table, new_refcount).

    ``table`` must hold every entry that owns a page. It and cache.refcount
    are left as they are, and stay readable until a page is written; to go on
    with the compacted pool, use new_table and copy new_refcount into
    cache.refcount."""
    _need(table, "table", torch.int32, 2)
    if out is None:
        new_table, new_refcount = torch.empty_like(table), torch.empty_like(cache.refcount)
    else:
        new_table, new_refcount = out
        _need(new_table, "new_table", torch.int32, 2)
        _need(new_refcount, "new_refcount", torch.int32, 1)
        if new_table.shape != table.shape or new_refcount.shape != cache.refcount.shape:
            raise ValueError("out must be (new_table [B,max_pages], new_refcount [num_pages])")
    _same_device(cache, table=table, new_table=new_table, new_refcount=new_refcount)
    ws = cache._workspace(workspace, 0)
    _finish(_lib.load().smla_cache_compact(cache._ref, _ptr(table), _ptr(new_table), _ptr(new_refcount),
                                           table.shape[0], table.shape[1], _ptr(ws), ws.numel(),
                                           _stream(cache.device)),
            "smla_cache_compact", ws, check_status)
    return new_table, new_refcount


def cache_copy_pages(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor,
                     workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Copy whole pages and their scales, src[i] to dst[i]. Every dst must differ from the others
    and from every src, else nothing is copied (smla_cache_copy_pages)."""
    _need(src, "src", torch.int32, 1)
    _need(dst, "dst", torch.int32, 1)
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    _same_device(cache, src=src, dst=dst)
    n = src.shape[0]
    ws = cache._workspace(workspace, n)
    _finish(_lib.load().smla_cache_copy_pages(cache._ref, _ptr(src), _ptr(dst), n, _ptr(ws), ws.numel(),
                                              _stream(cache.device)),
            "smla_cache_copy_pages", ws, check_status)
