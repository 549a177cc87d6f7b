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
from .api import D_HEAD, Workspace, _current_device, _need, device_status

# A decode step makes these calls once a layer, and their kernels take some ten
# microseconds: checks and marshalling are kept to a few attribute reads a tensor.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _check(cache: "PagedCache", t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> int:
    """Address of a tensor that a call can take; raises what _need raises, or for its device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.get_device() == cache._index
            and t.is_contiguous()):
        _need(t, name, dtype, ndim)
        raise ValueError(f"{name} must be on {cache.device}, got {t.device}")
    return t.data_ptr()


class PagedCache:
    """A pool of pages for the kv rows of many sequences.

    pages    [num_pages, page_size, 512] float8_e4m3fn
    scales   [num_pages, page_size // scale_block] float32: row value = code * scale
    refcount [num_pages] int32: table entries that hold the page (0: free)

    page_size is 16, 32, 64, 128 or 256, scale_block 16, 32 or 64. The tensors
    are the caller's: the handle keeps them and the C struct that names them. New
    contents are copied into them (after cache_compact, say); other tensors need another
    handle.
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
        self._pages, self._scales, self._refcount = pages, scales, refcount
        self.num_pages, self.page_size = n, ps
        self.scale_block = ps // scales.shape[1]
        self.device = pages.device
        self._index = pages.get_device()
        self._sizes = {}
        self._c = SmlaCache(pages=pages.data_ptr(), scales=scales.data_ptr(),
                            refcount=refcount.data_ptr(), num_pages=n, page_size=ps,
                            scale_block=self.scale_block, D=d)
        self._ref = ctypes.byref(self._c)
        self._lib = _lib.load()
        size = ctypes.c_size_t(0)
        _lib.check(self._lib.smla_cache_workspace_size(self._ref, 0, ctypes.byref(size)), "PagedCache")

    # (read-only: the calls go by the C struct, so another tensor put in place would not be seen)
    pages = property(lambda self: self._pages)
    scales = property(lambda self: self._scales)
    refcount = property(lambda self: self._refcount)

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
        size = self._sizes.get(n)
        if size is None:
            out = ctypes.c_size_t(0)
            _lib.check(_lib.load().smla_cache_workspace_size(self._ref, n, ctypes.byref(out)),
                       "smla_cache_workspace_size")
            size = self._sizes[n] = out.value
        return _on_device(self, workspace, size)


def _on_device(cache: PagedCache, workspace: Optional[Workspace], size: int) -> torch.Tensor:
    ws = (workspace or Workspace(cache.device)).get(size)
    if ws.get_device() != cache._index:
        raise ValueError(f"workspace must be on {cache.device}, got {ws.device}")
    return ws


def _check2(cache: "PagedCache", t: torch.Tensor, name: str, dtype: torch.dtype, n: int, m: int) -> int:
    """_check of a tensor of n x m."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (n, m) and t.get_device() == cache._index
            and t.is_contiguous()):
        return t.data_ptr()
    _check(cache, t, name, dtype, 2)
    raise ValueError(f"{name} must have shape [{n}, {m}], got {tuple(t.shape)}")


def _check1(cache: "PagedCache", t: torch.Tensor, name: str, dtype: torch.dtype, n: int) -> int:
    """_check of a vector of n."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (n,) and t.get_device() == cache._index
            and t.is_contiguous()):
        return t.data_ptr()
    _check(cache, t, name, dtype, 1)
    raise ValueError(f"{name} must have shape [{n}], got {tuple(t.shape)}")


def _size_of(sizes: dict, key, where: str, *args) -> int:
    """What the library's size query `where` says, asked once for each key."""
    size = sizes.get(key)
    if size is None:
        out = ctypes.c_size_t(0)
        _lib.check(getattr(_lib.load(), where)(*args, ctypes.byref(out)), where)
        size = sizes[key] = out.value
    return size


_paged_sizes = {}
_weights_sizes = {}
_reorder_sizes = {}


def _paged_size(dims: SmlaPagedDims) -> int:
    key = (dims.T > 0, dims.H)            # what smla_paged_workspace_size goes by
    size = _paged_sizes.get(key)
    if size is None:
        out = ctypes.c_size_t(0)
        _lib.check(_lib.load().smla_paged_workspace_size(ctypes.byref(dims), ctypes.byref(out)),
                   "smla_paged_workspace_size")
        size = _paged_sizes[key] = out.value
    return size


def _run(cache: PagedCache, where: str, ws: torch.Tensor, check_status: bool, *args) -> None:
    """Calls library function `where` with args, the workspace and the cache's device's stream."""
    fn = getattr(cache._lib, where)
    tail = (ws.data_ptr(), ws.numel(), _raw_stream(cache._index))
    if _current_device() == cache._index:
        code = fn(*args, *tail)
    else:
        with torch.cuda.device(cache._index):
            code = fn(*args, *tail)
    if code != _lib.SMLA_OK:
        raise _lib.SmlaError(code, where)
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
    (a padded slot: its seq and picks are not looked at) gets zeros. ``out`` =
    (o, lse) writes into the caller's tensors.
    """
    p_q = _check(cache, q, "q", torch.bfloat16, 3)
    p_table = _check(cache, table, "table", torch.int32, 2)
    p_lens = _check(cache, lens, "lens", torch.int32, 1)
    T, H, D = q.shape
    B, max_pages = table.shape
    if lens.shape[0] != T:
        raise ValueError("lens must have shape [T]")
    K = 0
    p_topk = p_seq = p_sink = None
    if topk is not None:
        p_topk = _check(cache, topk, "topk", torch.int32, 2)
        K = topk.shape[1]
        if topk.shape[0] != T or K < 1:
            raise ValueError("topk must have shape [T, K], K >= 1")
    if seq is not None:
        p_seq = _check(cache, seq, "seq", torch.int32, 1)
        if seq.shape[0] != T:
            raise ValueError("seq must have shape [T]")
    elif T > B:
        raise ValueError("without seq, table must have a row for each token")
    if sink is not None:
        p_sink = _check(cache, sink, "sink", torch.float32, 1)
        if sink.shape[0] != H:
            raise ValueError("sink must have shape [H]")
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((T, H), dtype=torch.float32, device=cache.device)
        p_o, p_lse = o.data_ptr(), lse.data_ptr()
    else:
        o, lse = out
        p_o = _check(cache, o, "o", torch.bfloat16, 3)
        p_lse = _check(cache, lse, "lse", torch.float32, 2)
        if o.shape != q.shape or tuple(lse.shape) != (T, H):
            raise ValueError("out must be (o [T,H,D], lse [T,H])")
    dims = SmlaPagedDims(T, H, D, K, B, max_pages, 0.0 if scale is None else float(scale))
    ws = _on_device(cache, workspace, _paged_size(dims))
    _run(cache, "smla_fwd_paged", ws, check_status, p_q, cache._ref, p_table, p_seq, p_lens, p_topk, p_sink, p_o,
         p_lse, ctypes.byref(dims))
    return o, lse


def cache_write(cache: PagedCache, table: torch.Tensor, start: torch.Tensor, cu_rows: torch.Tensor,
                rows: torch.Tensor, workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Write rows[cu_rows[b]:cu_rows[b+1]] (bf16 [n,512]) to the positions from start[b] on of
    the sequence in table row b, quantised block by block (smla_cache_write)."""
    p_table = _check(cache, table, "table", torch.int32, 2)
    p_start = _check(cache, start, "start", torch.int32, 1)
    p_cu = _check(cache, cu_rows, "cu_rows", torch.int32, 1)
    p_rows = _check(cache, rows, "rows", torch.bfloat16, 2)
    B = table.shape[0]
    if start.shape[0] != B or cu_rows.shape[0] != B + 1:
        raise ValueError("start must have shape [B] and cu_rows [B+1]")
    if rows.shape[1] != D_HEAD:
        raise ValueError("rows must have shape [n, 512]")
    _run(cache, "smla_cache_write", _on_device(cache, workspace, 256), check_status, cache._ref, p_table, p_start,
         p_cu, p_rows, B, table.shape[1], rows.shape[0])


def cache_alloc(cache: PagedCache, table: torch.Tensor, lens: torch.Tensor,
                workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Give every sequence the pages that lens[b] rows need, in place on table and
    cache.refcount; lowest free pages first, all or nothing (smla_cache_alloc)."""
    p_table = _check(cache, table, "table", torch.int32, 2)
    p_lens = _check(cache, lens, "lens", torch.int32, 1)
    B = table.shape[0]
    if lens.shape[0] != B:
        raise ValueError("lens must have shape [B]")
    _run(cache, "smla_cache_alloc", cache._workspace(workspace, B), check_status, cache._ref, p_table, p_lens, B,
         table.shape[1])


def cache_fork(cache: PagedCache, table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
               out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
               check_status: bool = True) -> torch.Tensor:
    """Fork sequences: the table rows [n, max_pages] of the children of rows parents[i].

    Full pages are shared (refcount + 1), a partly filled last page is copied
    to a free one. All or nothing. ``out`` takes the child rows."""
    p_table = _check(cache, table, "table", torch.int32, 2)
    p_lens = _check(cache, lens, "lens", torch.int32, 1)
    p_parents = _check(cache, parents, "parents", torch.int32, 1)
    B, max_pages = table.shape
    n = parents.shape[0]
    if lens.shape[0] != B:
        raise ValueError("lens must have shape [B]")
    child = table.new_empty((n, max_pages)) if out is None else out
    p_child = _check(cache, child, "out", torch.int32, 2)
    if tuple(child.shape) != (n, max_pages):
        raise ValueError("out must have shape [n, max_pages]")
    _run(cache, "smla_cache_fork", cache._workspace(workspace, n), check_status, cache._ref, p_table, p_lens,
         p_parents, p_child, B, n, max_pages)
    return child


def cache_free(cache: PagedCache, table: torch.Tensor, rows: Optional[torch.Tensor] = None,
               workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Give back the pages of the table rows listed in ``rows`` (all rows without it): their
    entries become -1 and the pages' refcounts fall by one (smla_cache_free)."""
    p_table = _check(cache, table, "table", torch.int32, 2)
    p_rows = None if rows is None else _check(cache, rows, "rows", torch.int32, 1)
    B = table.shape[0]
    n = B if rows is None else rows.shape[0]
    _run(cache, "smla_cache_free", _on_device(cache, workspace, 256), check_status, cache._ref, p_table, p_rows, B, n,
         table.shape[1])


def cache_compact(cache: PagedCache, table: torch.Tensor, workspace: Optional[Workspace] = None,
                  check_status: bool = True,
                  out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Move the last live pages into the holes before them: (new_table, new_refcount).

    ``table`` must hold every entry that owns a page. It and cache.refcount
    are left as they are, and stay readable until a page is written; to go on
    with the compacted pool, use new_table and copy new_refcount into
    cache.refcount."""
    p_table = _check(cache, table, "table", torch.int32, 2)
    if out is None:
        new_table, new_refcount = torch.empty_like(table), torch.empty_like(cache.refcount)
    else:
        new_table, new_refcount = out
    p_new = _check(cache, new_table, "new_table", torch.int32, 2)
    p_count = _check(cache, new_refcount, "new_refcount", torch.int32, 1)
    if new_table.shape != table.shape or new_refcount.shape != cache.refcount.shape:
        raise ValueError("out must be (new_table [B,max_pages], new_refcount [num_pages])")
    _run(cache, "smla_cache_compact", cache._workspace(workspace, 0), check_status, cache._ref, p_table, p_new,
         p_count, table.shape[0], table.shape[1])
    return new_table, new_refcount


def cache_copy_pages(cache: PagedCache, src: torch.Tensor, dst: torch.Tensor,
                     workspace: Optional[Workspace] = None, check_status: bool = True) -> None:
    """Copy whole pages and their scales, src[i] to dst[i]. Every dst must differ from the others
    and from every src, else nothing is copied (smla_cache_copy_pages)."""
    p_src = _check(cache, src, "src", torch.int32, 1)
    p_dst = _check(cache, dst, "dst", torch.int32, 1)
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    n = src.shape[0]
    _run(cache, "smla_cache_copy_pages", cache._workspace(workspace, n), check_status, cache._ref, p_src, p_dst, n)


def cache_weights(q: torch.Tensor, cache: PagedCache, table: torch.Tensor, lens: torch.Tensor, lse: torch.Tensor,
                  weights: torch.Tensor, cu_tokens: Optional[torch.Tensor] = None,
                  earlier: Optional[torch.Tensor] = None, decay: float = 1.0, scale: Optional[float] = None,
                  workspace: Optional[Workspace] = None, check_status: bool = True) -> torch.Tensor:
    """The attention weight that each cached position gets from query tokens, added up over them and their heads:
    weights = decay * earlier + sum of exp(scale <q, x> - lse) (smla_cache_weights). Returns ``weights``.

    q [T,H,512] bf16, lens [T] and lse [T,H] are those of sparse_mla_fwd_paged over all positions (the lse of a call
    with ``topk`` does not fit: the terms would be no weights); the tokens cu_tokens[b]:cu_tokens[b+1] belong to table
    row b (token b without it), so tokens come in the order of their sequences. weights and earlier are
    [B, max_pages * page_size] float32; without ``earlier`` the sums are added to ``weights`` itself. With decay 0
    nothing earlier counts. Positions that no token sees keep what ``weights`` has. T * H is at most 2^25.
    """
    p_q = _check(cache, q, "q", torch.bfloat16, 3)
    p_table = _check(cache, table, "table", torch.int32, 2)
    T, H, D = q.shape
    B, max_pages = table.shape
    width = max_pages * cache.page_size
    p_lens = _check1(cache, lens, "lens", torch.int32, T)
    p_lse = _check2(cache, lse, "lse", torch.float32, T, H)
    p_weights = _check2(cache, weights, "weights", torch.float32, B, width)
    p_cu, p_earlier = None, p_weights
    if cu_tokens is not None:
        p_cu = _check1(cache, cu_tokens, "cu_tokens", torch.int32, B + 1)
    elif T > B:
        raise ValueError("without cu_tokens, table must have a row for each token")
    if earlier is not None:
        p_earlier = _check2(cache, earlier, "earlier", torch.float32, B, width)
    dims = SmlaPagedDims(T, H, D, 0, B, max_pages, 0.0 if scale is None else float(scale))
    ws = _on_device(cache, workspace, _size_of(_weights_sizes, (T, H), "smla_weights_workspace_size", dims))
    _run(cache, "smla_cache_weights", ws, check_status, p_q, cache._ref, p_table, p_cu, p_lens, p_lse, p_earlier,
         decay, p_weights, ctypes.byref(dims))
    return weights


def cache_evict(cache: PagedCache, table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor, keep: int,
                first: int = 0, recent: int = 0, workspace: Optional[Workspace] = None, check_status: bool = True,
                out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]] = None
                ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Keep min(lens[b], keep) positions of every sequence, in fresh pages: the first ``first``, the last ``recent``
    and, of the others, those of largest weight (smla_cache_evict). Returns (new_table, new_lens, new_weights, kept);
    kept [B, keep] says which position each row had.

    weights [B, max_pages * page_size] float32 (cache_weights). The old sequences stay as they are: cache_free gives
    their pages back. All or nothing where free pages are short or a sequence has a page that nobody owns (refcount 0).
    ``out`` takes the four results.
    """
    p_table = _check(cache, table, "table", torch.int32, 2)
    B, max_pages = table.shape
    width = max_pages * cache.page_size
    p_lens = _check1(cache, lens, "lens", torch.int32, B)
    p_weights = _check2(cache, weights, "weights", torch.float32, B, width)
    keep, first, recent = int(keep), int(first), int(recent)
    if not 1 <= keep <= width or first < 0 or recent < 0 or first + recent > keep:
        raise ValueError("1 <= keep <= max_pages * page_size and first + recent <= keep are needed")
    if out is None:
        out = (torch.empty_like(table), torch.empty_like(lens), torch.empty_like(weights),
               torch.empty((B, keep), dtype=torch.int32, device=cache.device))
    new_table, new_lens, new_weights, kept = out
    p_new = _check2(cache, new_table, "new_table", torch.int32, B, max_pages)
    p_len = _check1(cache, new_lens, "new_lens", torch.int32, B)
    p_moved = _check2(cache, new_weights, "new_weights", torch.float32, B, width)
    p_kept = _check2(cache, kept, "kept", torch.int32, B, keep)
    size = _size_of(cache._sizes, ("evict", B, keep), "smla_cache_evict_workspace_size", cache._ref, B, keep)
    _run(cache, "smla_cache_evict", _on_device(cache, workspace, size), check_status, cache._ref, p_table, p_lens,
         p_weights, p_new, p_len, p_moved, p_kept, B, max_pages, keep, first, recent)
    return out


def cache_reorder(cache: PagedCache, table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
                  weights: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
                  check_status: bool = True,
                  out: Optional[Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Row i of the new table continues row parents[i] of ``table`` (-1: an empty row): (new_table [n, max_pages],
    new_lens [n], new_weights or None) (smla_cache_reorder).

    A row's first child takes it over, its other children share its full pages and get a copy of a partly filled
    last one, and rows without a child are given back: the old table is void afterwards, unless the call ran
    short of pages (all or nothing). With ``weights`` [B, max_pages * page_size] the accumulated weights go along.
    """
    p_table = _check(cache, table, "table", torch.int32, 2)
    p_parents = _check(cache, parents, "parents", torch.int32, 1)
    B, max_pages = table.shape
    n = parents.shape[0]
    p_lens = _check1(cache, lens, "lens", torch.int32, B)
    if out is None:
        out = (table.new_empty((n, max_pages)), lens.new_empty(n),
               None if weights is None else weights.new_empty((n, max_pages * cache.page_size)))
    new_table, new_lens, new_weights = out
    p_new = _check2(cache, new_table, "new_table", torch.int32, n, max_pages)
    p_len = _check1(cache, new_lens, "new_lens", torch.int32, n)
    p_weights = p_moved = None
    if weights is not None:
        p_weights = _check2(cache, weights, "weights", torch.float32, B, max_pages * cache.page_size)
        p_moved = _check2(cache, new_weights, "new_weights", torch.float32, n, max_pages * cache.page_size)
    elif new_weights is not None:
        raise ValueError("out must have None for the weights where none are given")
    size = _size_of(_reorder_sizes, (B, n), "smla_cache_reorder_workspace_size", B, n)
    _run(cache, "smla_cache_reorder", _on_device(cache, workspace, size), check_status, cache._ref, p_table, p_lens,
         p_parents, p_weights, p_new, p_len, p_moved, B, n, max_pages)
    return out
