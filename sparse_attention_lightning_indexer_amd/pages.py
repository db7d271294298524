"""Pages of the paged caches (``include/indexer_pages.h``).

The state of a pool lives on the GPU: refs i32 [n_pages], the holders of each
page (none: the page is free); block_table i32 [rows, columns], the pages of
each request, -1 where it has none; seq_lens i32 [rows].  ``pages_grow`` gives
requests pages and slots for new tokens (the slots ``mx4_cache_write`` takes),
``pages_fork`` starts requests as others are, sharing their pages,
``pages_free`` ends requests, ``pages_compact`` moves the pages in use to the
front and ``pages_copy`` copies pages.  Argument checks and marshalling only,
as in the rest of the binding.
"""
from __future__ import annotations

import ctypes
import struct

from . import mx4 as _mx4

PAGES_EXPORTS = ("indexer_pages_copy", "indexer_pages_fork", "indexer_pages_grow", "indexer_pages_free",
                 "indexer_pages_compact", "indexer_pages_compact_workspace_bytes")

# The structures of include/indexer_pages.h, member by member
ARRAY = struct.Struct("=3q")
COPY = struct.Struct("=4q3i4x")
FORK = struct.Struct("=9q6i")
GROW = struct.Struct("=8q6i")
FREE = struct.Struct("=6q4i")
COMPACT = struct.Struct("=9q4i")

_lib = None
_torch = None


def _library():
    global _lib, _torch
    if _lib is None:
        lib = _mx4._library()
        for name in PAGES_EXPORTS[:5]:
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.c_char_p], ctypes.c_int
        lib.indexer_pages_compact_workspace_bytes.argtypes = [ctypes.c_int32]
        lib.indexer_pages_compact_workspace_bytes.restype = ctypes.c_size_t
        _torch = _mx4._torch
        _lib = lib
    return _lib


class PageSet:
    """The caches of a model, checked and listed once for the calls that move pages.

    Each tensor is [n_pages, ...] of any type, every page's bytes without gaps
    (in any order of the other dimensions): the data and scale tensors of the
    4-bit cache (where K and V scales lie side by side, the tensor of both),
    the indexer's key cache, of all layers."""

    def __init__(self, tensors):
        _library()
        self.tensors = tuple(tensors)      # the caches live as long as their list
        if not self.tensors:
            raise ValueError("a PageSet needs at least one cache")
        listed = []
        for i, t in enumerate(self.tensors):
            dev = _mx4._gpu(t, f"cache {i}")
            if t.dim() < 1:
                raise ValueError(f"cache {i} must be [n_pages, ...]")
            if i == 0:
                self.device, self.n_pages = dev, t.shape[0]
            if dev != self.device:
                raise ValueError(f"cache {i} is on GPU {dev}, expected {self.device}")
            if t.shape[0] != self.n_pages:
                raise ValueError(f"cache {i} has {t.shape[0]} pages, expected {self.n_pages}")
            values = 1
            for stride, size in sorted((t.stride(d), t.shape[d]) for d in range(1, t.dim()) if t.shape[d] != 1):
                if stride != values and size:
                    raise ValueError(f"cache {i}'s pages must have no gaps")
                values *= size
            if values == 0:
                raise ValueError(f"cache {i}'s pages are empty")
            if self.n_pages:
                listed.append(ARRAY.pack(t.data_ptr(), t.stride(0) * t.element_size(), values * t.element_size()))
        self.n_arrays = len(listed)
        self._buffer = ctypes.create_string_buffer(b"".join(listed) or b"\0")
        self.address = ctypes.addressof(self._buffer)


def _set(pages):
    return pages if isinstance(pages, PageSet) else PageSet(pages)


def _ints(t, name, dev, n=None):
    """Checks a contiguous i32 vector; its length."""
    if not (isinstance(t, _torch.Tensor) and t.dtype is _torch.int32 and t.get_device() == dev and t.dim() == 1
            and t.is_contiguous()):
        _mx4._need(t, name, _torch.int32, dev, 1)
        raise ValueError(f"{name} must be contiguous")
    size = t.shape[0]
    if n is not None and size != n:
        raise ValueError(f"{name} must have {n} entries, got {size}")
    return size


def _table(block_table, dev):
    """(rows, columns, row stride) of a block table."""
    if not (isinstance(block_table, _torch.Tensor) and block_table.dtype is _torch.int32
            and block_table.get_device() == dev and block_table.dim() == 2):
        _mx4._need(block_table, "block_table", _torch.int32, dev, 2)
    rows, cols = block_table.shape
    stride, one = block_table.stride()
    if cols > 1 and one != 1:
        raise ValueError("block_table rows must be contiguous")
    return rows, cols, stride if rows > 1 else cols


def _refs(refs):
    """(device, pages) of the counts, which every state has."""
    dev = _mx4._gpu(refs, "refs")
    return dev, _ints(refs, "refs", dev)


def pages_copy(pages, source, target) -> None:
    """Page source[i] of every cache to page target[i] (i32; a pair with either
    outside the pool is skipped).  pages: a PageSet, or the caches.  No page is
    named twice in target, or in both."""
    lib = _library()
    pages = _set(pages)
    dev = pages.device
    n = _ints(source, "source", dev)
    _ints(target, "target", dev, n)
    if n == 0:
        return
    _mx4._call(dev, lib.indexer_pages_copy, _mx4._pack(
        COPY, pages.address, source.data_ptr(), target.data_ptr(), _mx4._stream(dev), pages.n_arrays, n, pages.n_pages))


def pages_fork(pages, refs, block_table, seq_lens, parents, children, block_size: int, fresh=None):
    """Requests children[i] (rows of the table) begin as requests parents[i]
    are: they share the parents' full pages and get a copy of the last, partly
    filled one.  -> fresh i32 [n]: the page of the copy, -1 none needed (or the
    parent's is not of the pool, then the child has none either), -2 none free
    (the child is empty), -3 skipped (a row that is not there, or a child named
    before).  What a child held is overwritten: free it first.
    pages None: no bytes are copied."""
    lib = _library()
    dev, n_pages = _refs(refs)
    if pages is not None:
        pages = _set(pages)
        if pages.device != dev or pages.n_pages != n_pages:
            raise ValueError(f"refs must have one count per page ({pages.n_pages}) on GPU {pages.device}")
    rows, cols, stride = _table(block_table, dev)
    _ints(seq_lens, "seq_lens", dev, rows)
    n = _ints(parents, "parents", dev)
    _ints(children, "children", dev, n)
    if fresh is None:
        fresh = parents.new_empty(n)
    else:
        _ints(fresh, "fresh", dev, n)
    if n == 0:
        return fresh
    _mx4._call(dev, lib.indexer_pages_fork, _mx4._pack(
        FORK, pages.address if pages else 0, refs.data_ptr(), block_table.data_ptr(), stride, seq_lens.data_ptr(),
        parents.data_ptr(), children.data_ptr(), fresh.data_ptr(), _mx4._stream(dev), pages.n_arrays if pages else 0, n,
        n_pages, rows, cols, block_size))
    return fresh


def pages_grow(refs, block_table, seq_lens, rows, tokens: int, block_size: int, new_tokens=None, slots=None):
    """Requests rows[i] get `tokens` more tokens, or new_tokens[i] (i32, at
    most `tokens`) of them: free pages, lowest first, in the order of the list,
    and their lengths.  -> slots i64 [n, tokens], -1 past a request's new
    tokens and for requests that could not grow (no free page or no column
    left, or a last page that is not of the pool; they stay as they were) or
    were skipped."""
    lib = _library()
    dev, n_pages = _refs(refs)
    n_rows, cols, stride = _table(block_table, dev)
    _ints(seq_lens, "seq_lens", dev, n_rows)
    n = _ints(rows, "rows", dev)
    if new_tokens is not None:
        _ints(new_tokens, "new_tokens", dev, n)
    if tokens < 0:
        raise ValueError(f"tokens={tokens} must be >= 0")
    if slots is None:
        slots = refs.new_empty((n, tokens), dtype=_torch.int64)
    else:
        _mx4._need(slots, "slots", _torch.int64, dev, 2)
        if slots.shape != (n, tokens) or not slots.is_contiguous():
            raise ValueError(f"slots must be contiguous [{n}, {tokens}]")
    if n == 0 or tokens == 0:
        return slots
    _mx4._call(dev, lib.indexer_pages_grow, _mx4._pack(
        GROW, refs.data_ptr(), block_table.data_ptr(), stride, seq_lens.data_ptr(), rows.data_ptr(),
        0 if new_tokens is None else new_tokens.data_ptr(), slots.data_ptr(), _mx4._stream(dev), n, tokens, n_pages,
        n_rows, cols, block_size))
    return slots


def pages_free(refs, block_table, seq_lens, rows) -> None:
    """Requests rows[i] end: the pages they hold have one holder less, their
    table rows become -1, their lengths 0."""
    lib = _library()
    dev, n_pages = _refs(refs)
    n_rows, cols, stride = _table(block_table, dev)
    _ints(seq_lens, "seq_lens", dev, n_rows)
    n = _ints(rows, "rows", dev)
    if n == 0 or n_rows == 0:
        return
    _mx4._call(dev, lib.indexer_pages_free, _mx4._pack(
        FREE, refs.data_ptr(), block_table.data_ptr(), stride, seq_lens.data_ptr(), rows.data_ptr(), _mx4._stream(dev), n,
        n_pages, n_rows, cols))


def pages_compact(pages, refs, block_table, place=None, live=None, workspace=None):
    """The pages in use, L of them, moved to the pages below L: bytes of every
    cache, refs and the table's entries.  -> (place i32 [n_pages]: where each
    page went, -1 for free ones; live i32 [1]: L).  pages None: no bytes."""
    lib = _library()
    dev, n_pages = _refs(refs)
    if pages is not None:
        pages = _set(pages)
        if pages.device != dev or pages.n_pages != n_pages:
            raise ValueError(f"refs must have one count per page ({pages.n_pages}) on GPU {pages.device}")
    rows, cols, stride = _table(block_table, dev)
    if place is None:
        place = refs.new_empty(n_pages)
    else:
        _ints(place, "place", dev, n_pages)
    if live is None:
        live = refs.new_empty(1)
    else:
        _ints(live, "live", dev, 1)
    if workspace is None:
        workspace = refs.new_empty(int(lib.indexer_pages_compact_workspace_bytes(n_pages)), dtype=_torch.uint8)
    else:
        _mx4._need(workspace, "workspace", _torch.uint8, dev, 1)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _mx4._call(dev, lib.indexer_pages_compact, _mx4._pack(
        COMPACT, pages.address if pages else 0, refs.data_ptr(), block_table.data_ptr(), stride, place.data_ptr(),
        live.data_ptr(), workspace.data_ptr(), workspace.numel(), _mx4._stream(dev), pages.n_arrays if pages else 0,
        n_pages, rows, cols))
    return place, live


def pages_compact_workspace_bytes(n_pages: int) -> int:
    """Workspace of a compaction."""
    if not 0 <= n_pages < 2**31:
        raise ValueError(f"n_pages={n_pages} is not a number of pages")
    return int(_library().indexer_pages_compact_workspace_bytes(n_pages))
