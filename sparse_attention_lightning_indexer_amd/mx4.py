"""The 4-bit key/value cache and the attention over it (``include/indexer_mx4.h``).

What follows the selection: ``mx4_cache_write`` quantises a step's or a prompt's
keys and values into a paged cache in microscaled 4-bit floats,
``mx4_cache_read`` gives rows back as numbers, ``mx4_attend_selected`` attends
to the keys a top-k selected and ``mx4_attend_window`` to a sliding window with
a few first tokens.  Argument checks and marshalling only, as in the rest of
the binding: the work is in the library's HIP kernels, on torch's current
stream of the tensors' device.

A cache is a pair of uint8 tensors, data ``[n_blocks, block_size, n_heads,
head_dim/2]`` and scale ``[n_blocks, block_size, n_heads, head_dim/32]``; block,
slot and head may be strided in any order (a permuted view of
``[n_blocks, n_heads, block_size, ...]`` works), the last dimension contiguous.
"""
from __future__ import annotations

import ctypes
import sys
from typing import Optional, Tuple

_pkg = sys.modules[__package__]

MX4_EXPORTS = (
    "indexer_mx4_cache_write", "indexer_mx4_cache_read", "indexer_mx4_attend_selected",
    "indexer_mx4_attend_window", "indexer_mx4_attend_workspace_bytes",
)
MX4_F16, MX4_BF16 = 0, 1
MAX_KEYS = 2**31 - 1024

_ready = None


def _library():
    """The library with these entry points' signatures declared."""
    global _ready
    lib = _pkg.load_library()
    if _ready is lib:
        return lib
    p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    pages = [i32, i32] + [i64] * 6
    cached = [p, i64, i64, i32, p, p, p, p] + pages + [p, i64, p] + [i32] * 6 + [ctypes.c_float]
    out = [p, i64, i64, p, p, sz, p]
    lib.indexer_mx4_cache_write.argtypes = [p, i64, i64, p, i64, i64, i32, i32, i32, i32, p, p, p, p, p] + pages + [p]
    lib.indexer_mx4_cache_read.argtypes = [p, p] + pages + [p, i32, i32, i32, p, i64, i64, i32, p]
    lib.indexer_mx4_attend_selected.argtypes = cached + [p, i64, i32, i32] + out
    lib.indexer_mx4_attend_window.argtypes = cached + [i32, i32] + out
    for f in (lib.indexer_mx4_cache_write, lib.indexer_mx4_cache_read, lib.indexer_mx4_attend_selected,
              lib.indexer_mx4_attend_window):
        f.restype = ctypes.c_int
    lib.indexer_mx4_attend_workspace_bytes.argtypes = [i32] * 7
    lib.indexer_mx4_attend_workspace_bytes.restype = sz
    _ready = lib
    return lib


def _type_of(dtype) -> int:
    torch = _pkg._torch()
    if dtype == torch.float16:
        return MX4_F16
    if dtype == torch.bfloat16:
        return MX4_BF16
    raise TypeError(f"the 4-bit cache takes torch.float16 or torch.bfloat16, got {dtype}")


def _rows(t, name, dtype, device, shape=None):
    """Rows [n, heads, d] with d contiguous."""
    _pkg._need(t, name, dtype, device, 3)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _stride(t, dim, natural):
    """A dimension's stride in elements; that of one entry says nothing."""
    return t.stride(dim) if t.shape[dim] > 1 else natural


def _row_strides(t):
    """Row and head strides of [n, heads, d] rows."""
    sh = _stride(t, 1, t.shape[2])
    return _stride(t, 0, t.shape[1] * max(sh, t.shape[2])), sh


def _cache(data, scale, name, device, heads, d):
    """Checks one cache; its (n_blocks, block_size, strides in bytes)."""
    torch = _pkg._torch()
    _pkg._need(data, f"{name}_data", torch.uint8, device, 4)
    _pkg._need(scale, f"{name}_scale", torch.uint8, device, 4)
    blocks, size = data.shape[0], data.shape[1]
    if d % 32 or tuple(data.shape[2:]) != (heads, d // 2):
        raise ValueError(f"{name}_data must be [n_blocks, block_size, {heads}, {d}/2] (head_dim a multiple of 32), got "
                         f"{list(data.shape)}")
    if tuple(scale.shape) != (blocks, size, heads, d // 32):
        raise ValueError(f"{name}_scale must be {[blocks, size, heads, d // 32]}, got {list(scale.shape)}")
    if data.stride(3) != 1 or (scale.stride(3) != 1 and d > 32):
        raise ValueError(f"{name}_data's and {name}_scale's last dimension must be contiguous")
    return (blocks, size) + tuple(_stride(t, i, t.shape[3]) for t in (data, scale) for i in range(3))


def _slots(slots, n, device):
    _pkg._need(slots, "slots", _pkg._torch().int64, device, 1)
    if slots.shape[0] != n:
        raise ValueError(f"slots must have one entry per row ({n}), got {slots.shape[0]}")
    if n > 1 and slots.stride(0) != 1:
        raise ValueError("slots must be contiguous")


def _on(device):
    """Makes the tensors' device current for a launch, where it is not."""
    torch = _pkg._torch()
    return torch.cuda.device(device)


def _call(device, status_of):
    torch = _pkg._torch()
    if device.index is None or device.index == torch.cuda.current_device():
        _pkg._check(status_of())
    else:
        with _on(device):
            _pkg._check(status_of())


def mx4_cache_write(k, slots, k_data, k_scale, v=None, v_data=None, v_scale=None) -> None:
    """Quantise rows k (and v) [n_tokens, n_heads, d], f16 or bf16, into the
    cache: token t goes to slot slots[t] (i64; block * block_size + offset), a
    negative slot or one past the cache is skipped.  Slots that are not skipped
    must be distinct.  Every other slot keeps its bytes."""
    lib = _library()
    torch = _pkg._torch()
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise ValueError("k must be a GPU tensor")
    dev = k.device
    kind = _type_of(k.dtype)
    _rows(k, "k", k.dtype, dev)
    n, heads, d = k.shape
    pages = _cache(k_data, k_scale, "k", dev, heads, d)
    _slots(slots, n, dev)
    if (v is None) != (v_data is None) or (v is None) != (v_scale is None):
        raise ValueError("v, v_data and v_scale come together")
    if v is not None:
        _rows(v, "v", k.dtype, dev, k.shape)
        if _cache(v_data, v_scale, "v", dev, heads, d) != pages:
            raise ValueError("the K and V caches must have the same shape and strides")
    if n == 0 or pages[0] == 0:  # nothing to write, or nowhere (and empty tensors have no address)
        return
    ptr = _pkg._ptr
    _call(dev, lambda: lib.indexer_mx4_cache_write(
        ptr(k), *_row_strides(k), ptr(v), *(_row_strides(v) if v is not None else (0, 0)), kind, n, heads, d, ptr(slots), ptr(k_data), ptr(k_scale), ptr(v_data),
        ptr(v_scale), *pages, _pkg._stream(dev)))


def mx4_cache_read(data, scale, slots, dtype=None, out=None):
    """Rows of one cache (K or V) as numbers: [n_rows, n_heads, d] of `dtype`
    (float16 unless given, or out's), row i from slot slots[i] (zeros where
    that is negative or past the cache; a slot may come again)."""
    lib = _library()
    torch = _pkg._torch()
    if not isinstance(data, torch.Tensor) or not data.is_cuda:
        raise ValueError("data must be a GPU tensor")
    dev = data.device
    if data.dim() != 4:
        raise ValueError(f"data must have 4 dims, got {data.dim()}")
    heads, d = data.shape[2], 2 * data.shape[3]
    if dtype is None:
        dtype = torch.float16 if out is None else out.dtype
    kind = _type_of(dtype)
    pages = _cache(data, scale, "k", dev, heads, d)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a vector of slots")
    n = slots.shape[0]
    _slots(slots, n, dev)
    if out is None:
        out = torch.empty((n, heads, d), dtype=dtype, device=dev)
    _rows(out, "out", dtype, dev, (n, heads, d))
    if out.numel() == 0:
        return out
    if pages[0] == 0:  # an empty cache has no slot, and no address
        return out.zero_()
    ptr = _pkg._ptr
    _call(dev, lambda: lib.indexer_mx4_cache_read(
        ptr(data), ptr(scale), *pages, ptr(slots), n, heads, d, ptr(out), *_row_strides(out), kind,
        _pkg._stream(dev)))
    return out


def mx4_attend_workspace_bytes(n_requests: int, query_len: int, max_keys: int, selected: bool, n_heads: int,
                               n_kv_heads: int, head_dim: int) -> int:
    """Workspace of an attention call (see include/indexer_mx4.h for max_keys)."""
    return int(_library().indexer_mx4_attend_workspace_bytes(n_requests, query_len, max_keys, int(selected), n_heads,
                                                             n_kv_heads, head_dim))


def _attend(entry, q, k_data, k_scale, v_data, v_scale, block_table, seq_lens, query_len, max_seq_len, sm_scale,
            selected, max_keys, form, out, lse, with_lse, workspace):
    torch = _pkg._torch()
    lib = _library()
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    dev = q.device
    kind = _type_of(q.dtype)
    _rows(q, "q", q.dtype, dev)
    rows, heads, d = q.shape
    if not isinstance(k_data, torch.Tensor) or k_data.dim() != 4:
        raise ValueError("k_data must be [n_blocks, block_size, n_kv_heads, head_dim/2]")
    kv = k_data.shape[2]
    pages = _cache(k_data, k_scale, "k", dev, kv, d)
    if _cache(v_data, v_scale, "v", dev, kv, d) != pages:
        raise ValueError("the K and V caches must have the same shape and strides")
    _pkg._need(block_table, "block_table", torch.int32, dev, 2)
    _pkg._need(seq_lens, "seq_lens", torch.int32, dev, 1)
    requests = seq_lens.shape[0]
    if requests > 1 and seq_lens.stride(0) != 1:
        raise ValueError("seq_lens must be contiguous")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    if block_table.shape[0] < requests or block_table.shape[1] * pages[1] < max_seq_len:
        raise ValueError(f"block_table must be at least [n_requests, ceil(max_seq_len/block_size)] = [{requests}, "
                         f"{-(-max_seq_len // max(pages[1], 1))}], got {list(block_table.shape)}")
    if rows != requests * query_len:
        raise ValueError(f"q has {rows} rows, expected n_requests*query_len = {requests * query_len}")
    if out is None:
        out = torch.empty((rows, heads, d), dtype=q.dtype, device=dev)
    _rows(out, "out", q.dtype, dev, q.shape)
    if lse is None and with_lse:
        lse = torch.empty((rows, heads), dtype=torch.float32, device=dev)
    if lse is not None:
        _pkg._need(lse, "lse", torch.float32, dev, 2)
        if tuple(lse.shape) != (rows, heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{rows}, {heads}]")
    if rows == 0:  # nothing to compute
        return out, lse
    need = lib.indexer_mx4_attend_workspace_bytes(requests, query_len, max_keys, selected, heads, kv, d)
    if workspace is not None:
        _pkg._need(workspace, "workspace", torch.uint8, dev, 1)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    elif 0 < need < 2**63:  # sizes the library refuses have none: the call below names them
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ptr = _pkg._ptr
    _call(dev, lambda: getattr(lib, entry)(
        ptr(q), *_row_strides(q), kind, ptr(k_data), ptr(k_scale), ptr(v_data), ptr(v_scale), *pages,
        ptr(block_table), _stride(block_table, 0, block_table.shape[1]), ptr(seq_lens), requests, query_len, max_seq_len, heads, kv, d,
        sm_scale, *form, ptr(out), *_row_strides(out), ptr(lse), ptr(workspace),
        workspace.numel() if workspace is not None else 0, _pkg._stream(dev)))
    return out, lse


def mx4_attend_selected(q, k_data, k_scale, v_data, v_scale, block_table, seq_lens, query_len: int, idx,
                        sm_scale: float, pool_size: int = 1, out=None, lse=None, with_lse: bool = True,
                        workspace=None) -> Tuple:
    """Attention of each query row to the keys its selection names.

    q f16 or bf16 [R*Q, n_heads, d] (row r*Q+j is query j of request r, which
    sees keys s < seq_lens[r] - Q + 1 + j), idx i32 [R*Q, k] as the top-k
    gives it (-1: none; an entry stands for pool_size consecutive keys), the
    cache's four tensors, block_table i32 [R, max_blocks], seq_lens i32 [R]
    -> (out like q, lse f32 [R*Q, n_heads] or None).  Keys past the block
    table's pages are not seen.  A row with no key has out 0 and lse -inf."""
    torch = _pkg._torch()
    if not isinstance(q, torch.Tensor) or not isinstance(idx, torch.Tensor):
        raise TypeError("q and idx must be torch.Tensors")
    _pkg._need(idx, "idx", torch.int32, q.device, 2)
    if idx.shape[0] != q.shape[0]:
        raise ValueError(f"idx must have one row per row of q ({q.shape[0]}), got {idx.shape[0]}")
    if idx.shape[1] > 1 and idx.stride(1) != 1:
        raise ValueError("idx rows must be contiguous")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [n_requests, max_blocks]")
    if not isinstance(k_data, torch.Tensor) or k_data.dim() != 4:
        raise ValueError("k_data must be [n_blocks, block_size, n_kv_heads, head_dim/2]")
    if pool_size < 1:
        raise ValueError("pool_size must be >= 1")
    max_seq_len = min(block_table.shape[1] * k_data.shape[1], MAX_KEYS)
    n_sel = idx.shape[1]
    # an empty selection has no address: one entry of -1 attends to as little
    if n_sel == 0 and idx.shape[0] > 0:
        idx = torch.full((idx.shape[0], 1), -1, dtype=torch.int32, device=q.device)
        n_sel = 1
    return _attend("indexer_mx4_attend_selected", q, k_data, k_scale, v_data, v_scale, block_table, seq_lens,
                   query_len, max_seq_len, sm_scale, 1, min(n_sel * pool_size, 2**31 - 1),
                   (_pkg._ptr(idx), _stride(idx, 0, n_sel), n_sel, pool_size), out, lse, with_lse, workspace)


def mx4_attend_window(q, k_data, k_scale, v_data, v_scale, block_table, seq_lens, query_len: int, max_seq_len: int,
                      sm_scale: float, window: int = 0, sinks: int = 0, out=None, lse=None, with_lse: bool = True,
                      workspace=None) -> Tuple:
    """Attention of each query row to its last `window` keys and the first
    `sinks` tokens (window 0: every key it sees): with v = seq_lens[r] - Q + 1
    + j, the keys s < min(v, max_seq_len) that have s >= v - window or
    s < sinks.  Other arguments and results as in mx4_attend_selected."""
    keys = max_seq_len if window == 0 else min(max_seq_len, window + sinks)
    return _attend("indexer_mx4_attend_window", q, k_data, k_scale, v_data, v_scale, block_table, seq_lens, query_len,
                   max_seq_len, sm_scale, 0, max(0, min(keys, 2**31 - 1)), (window, sinks), out, lse, with_lse,
                   workspace)
