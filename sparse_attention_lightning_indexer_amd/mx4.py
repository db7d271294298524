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
import struct
import sys
from typing import Optional, Tuple

_pkg = sys.modules[__package__]

MX4_EXPORTS = (
    "indexer_mx4_cache_write", "indexer_mx4_cache_read", "indexer_mx4_attend_selected",
    "indexer_mx4_attend_window", "indexer_mx4_attend_workspace_bytes",
)
MX4_F16, MX4_BF16 = 0, 1
MAX_KEYS = 2**31 - 1024

# The argument structures of include/indexer_mx4.h, member by member: packing
# one is several times quicker than passing 40 arguments through ctypes
WRITE = struct.Struct("=18q6i")
READ = struct.Struct("=13q6i")
ATTEND = struct.Struct("=25q13if")

_lib = None        # the library with these entry points' signatures declared
_torch = None
_types = {}        # torch dtype -> the library's type code


def _library():
    global _lib, _torch
    if _lib is not None:
        return _lib
    lib = _pkg.load_library()
    for name in MX4_EXPORTS[:4]:
        f = getattr(lib, name)
        f.argtypes, f.restype = [ctypes.c_char_p], ctypes.c_int   # a packed argument structure
    lib.indexer_mx4_attend_workspace_bytes.argtypes = [ctypes.c_int32] * 7
    lib.indexer_mx4_attend_workspace_bytes.restype = ctypes.c_size_t
    if _torch is None:
        _torch = _pkg._torch()
        _types.update({_torch.float16: MX4_F16, _torch.bfloat16: MX4_BF16})
    _lib = lib
    return lib


# These calls are short, so the checks are: one test of everything that is
# usually right, and the framework's own check, which names what is not.

def _need(t, name, dtype, dev, dims):
    if not (isinstance(t, _torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == dims):
        _pkg._need(t, name, dtype, _torch.device("cuda", dev), dims)


def _gpu(t, name):
    """The index of the tensor's GPU."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.get_device()


def _type_of(dtype) -> int:
    kind = _types.get(dtype)
    if kind is None:
        raise TypeError(f"the 4-bit cache takes torch.float16 or torch.bfloat16, got {dtype}")
    return kind


def _rows(t, name, dtype, dev, shape=None):
    """Checks rows [n, heads, d] with d contiguous; their row and head strides
    (a dimension of one entry has whatever stride is natural)."""
    _need(t, name, dtype, dev, 3)
    n, heads, d = t.shape
    if shape is not None and (n, heads, d) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {[n, heads, d]}")
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if heads <= 1:
        sh = d
    return (st if n > 1 else heads * max(sh, d)), sh


def _cache(data, scale, of, dev, heads, d):
    """Checks one cache, whose arguments' names begin with `of`; its (n_blocks,
    block_size, strides in bytes)."""
    uint8 = _torch.uint8
    _need(data, of + "data", uint8, dev, 4)
    _need(scale, of + "scale", uint8, dev, 4)
    blocks, size, h, w = data.shape
    if d % 32 or h != heads or 2 * w != d:
        raise ValueError(f"{of}data must be [n_blocks, block_size, {heads}, {d}/2] (head_dim a multiple of 32), got "
                         f"{list(data.shape)}")
    if scale.shape != (blocks, size, heads, d // 32):
        raise ValueError(f"{of}scale must be {[blocks, size, heads, d // 32]}, got {list(scale.shape)}")
    db, ds, dh, one = data.stride()
    sb, ss, sh, sone = scale.stride()
    if one != 1 or (sone != 1 and d > 32):
        raise ValueError(f"{of}data's and {of}scale's last dimension must be contiguous")
    # a dimension of one entry: its stride says nothing
    if heads == 1:
        dh, sh = w, d // 32
    if size <= 1:
        ds, ss = w, d // 32
    if blocks <= 1:
        db, sb = w, d // 32
    return blocks, size, db, ds, dh, sb, ss, sh


def _like(data, scale, k_data, k_scale, dev):
    """Whether V's cache is as K's, which was checked."""
    tensor, uint8 = _torch.Tensor, _torch.uint8
    return (isinstance(data, tensor) and isinstance(scale, tensor) and data.dtype is uint8 and scale.dtype is uint8
            and data.get_device() == dev and scale.get_device() == dev and data.shape == k_data.shape
            and scale.shape == k_scale.shape and data.stride() == k_data.stride()
            and scale.stride() == k_scale.stride())


def _slots(slots, n, dev):
    _need(slots, "slots", _torch.int64, dev, 1)
    if slots.shape[0] != n:
        raise ValueError(f"slots must have one entry per row ({n}), got {slots.shape[0]}")
    if n > 1 and slots.stride(0) != 1:
        raise ValueError("slots must be contiguous")


def _pack(layout, *members):
    try:
        return layout.pack(*members)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"an argument is out of its range: {e}") from None


def _stream(dev):
    return _torch._C._cuda_getCurrentRawStream(dev)


def _call(dev, entry, args):
    """Calls the library with the tensors' device current."""
    if dev == _torch._C._cuda_getDevice():
        status = entry(args)
    else:
        with _torch.cuda.device(dev):
            status = entry(args)
    if status:
        _pkg._check(status)


def mx4_cache_write(k, slots, k_data, k_scale, v=None, v_data=None, v_scale=None) -> None:
    """Quantise rows k (and v) [n_tokens, n_heads, d], f16 or bf16, into the
    cache: token t goes to slot slots[t] (i64; block * block_size + offset), a
    negative slot or one past the cache is skipped.  Slots that are not skipped
    must be distinct.  Every other slot keeps its bytes."""
    lib = _library()
    dev = _gpu(k, "k")
    kind = _type_of(k.dtype)
    k_strides = _rows(k, "k", k.dtype, dev)
    n, heads, d = shape = tuple(k.shape)
    pages = _cache(k_data, k_scale, "k_", dev, heads, d)
    _slots(slots, n, dev)
    v_args, v_strides = (0, 0), (0, 0)
    if v is not None and v_data is not None and v_scale is not None:
        v_strides = _rows(v, "v", k.dtype, dev, shape)
        if not _like(v_data, v_scale, k_data, k_scale, dev) and _cache(v_data, v_scale, "v_", dev, heads, d) != pages:
            raise ValueError("the K and V caches must have the same shape and strides")
        v_args = (v_data.data_ptr(), v_scale.data_ptr())
    elif v is not None or v_data is not None or v_scale is not None:
        raise ValueError("v, v_data and v_scale come together")
    if n == 0 or pages[0] == 0:  # nothing to write, or nowhere (and empty tensors have no address)
        return
    blocks, size, *strides = pages
    _call(dev, lib.indexer_mx4_cache_write, _pack(
        WRITE, k.data_ptr(), *k_strides, 0 if v is None else v.data_ptr(), *v_strides, slots.data_ptr(),
        k_data.data_ptr(), k_scale.data_ptr(), *v_args, *strides, _stream(dev), kind, n, heads, d, blocks, size))


def mx4_cache_read(data, scale, slots, dtype=None, out=None):
    """Rows of one cache (K or V) as numbers: [n_rows, n_heads, d] of `dtype`
    (float16 unless given, or out's), row i from slot slots[i] (zeros where
    that is negative or past the cache; a slot may come again)."""
    lib = _library()
    dev = _gpu(data, "data")
    if data.dim() != 4:
        raise ValueError(f"data must have 4 dims, got {data.dim()}")
    heads, d = data.shape[2], 2 * data.shape[3]
    if dtype is None:
        dtype = _torch.float16 if out is None else out.dtype
    kind = _type_of(dtype)
    pages = _cache(data, scale, "", dev, heads, d)
    if not isinstance(slots, _torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a vector of slots")
    n = slots.shape[0]
    _slots(slots, n, dev)
    if out is None:
        out = data.new_empty((n, heads, d), dtype=dtype)
    strides = _rows(out, "out", dtype, dev, (n, heads, d))
    if n == 0 or heads == 0 or d == 0:
        return out
    if pages[0] == 0:  # an empty cache has no slot, and no address
        return out.zero_()
    blocks, size, *page_strides = pages
    _call(dev, lib.indexer_mx4_cache_read, _pack(
        READ, data.data_ptr(), scale.data_ptr(), *page_strides, slots.data_ptr(), out.data_ptr(), *strides,
        _stream(dev), kind, n, heads, d, blocks, size))
    return out


def mx4_attend_workspace_bytes(n_requests: int, query_len: int, max_keys: int, selected: bool, n_heads: int,
                               n_kv_heads: int, head_dim: int) -> int:
    """Workspace of an attention call (see include/indexer_mx4.h for max_keys;
    more than 2^31 - 1 of them count as that)."""
    sizes = (n_requests, query_len, min(max_keys, 2**31 - 1), int(bool(selected)), n_heads, n_kv_heads, head_dim)
    if not all(-2**31 <= n < 2**31 for n in sizes):   # ctypes would take their low 32 bits
        raise ValueError(f"sizes out of the 32-bit range: {sizes}")
    return int(_library().indexer_mx4_attend_workspace_bytes(*sizes))


def _attend(entry, q, k_data, k_scale, v_data, v_scale, block_table, seq_lens, query_len, max_seq_len, sm_scale,
            selected, max_keys, form, out, lse, with_lse, workspace):
    torch = _torch
    dev = _gpu(q, "q")
    dtype = q.dtype
    kind = _type_of(dtype)
    q_strides = _rows(q, "q", dtype, dev)
    rows, heads, d = shape = tuple(q.shape)
    if not isinstance(k_data, torch.Tensor) or k_data.dim() != 4:
        raise ValueError("k_data must be [n_blocks, block_size, n_kv_heads, head_dim/2]")
    kv = k_data.shape[2]
    pages = _cache(k_data, k_scale, "k_", dev, kv, d)
    if not _like(v_data, v_scale, k_data, k_scale, dev) and _cache(v_data, v_scale, "v_", dev, kv, d) != pages:
        raise ValueError("the K and V caches must have the same shape and strides")
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(seq_lens, "seq_lens", torch.int32, dev, 1)
    requests = seq_lens.shape[0]
    if requests > 1 and seq_lens.stride(0) != 1:
        raise ValueError("seq_lens must be contiguous")
    bt_rows, bt_cols = block_table.shape
    bt_stride, bt_one = block_table.stride()
    if bt_cols > 1 and bt_one != 1:
        raise ValueError("block_table rows must be contiguous")
    if bt_rows < requests or bt_cols * pages[1] < max_seq_len:
        raise ValueError(f"block_table must be at least [n_requests, ceil(max_seq_len/block_size)] = [{requests}, "
                         f"{-(-max_seq_len // max(pages[1], 1))}], got {[bt_rows, bt_cols]}")
    if rows != requests * query_len:
        raise ValueError(f"q has {rows} rows, expected n_requests*query_len = {requests * query_len}")
    if out is None:
        out = q.new_empty(shape)
        out_strides = (heads * d, d)
    else:
        out_strides = _rows(out, "out", dtype, dev, shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev, 2)
        if lse.shape != (rows, heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{rows}, {heads}]")
    elif with_lse:
        lse = q.new_empty((rows, heads), dtype=torch.float32)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev, 1)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    if rows == 0:  # nothing to compute
        return out, lse
    if workspace is None:
        need = _lib.indexer_mx4_attend_workspace_bytes(requests, query_len, max_keys, selected, heads, kv, d)
        if 0 < need < 2**63:  # sizes the library refuses have none: the call below names them
            workspace = q.new_empty(need, dtype=torch.uint8)
    blocks, size, *strides = pages
    _call(dev, entry, _pack(
        ATTEND, q.data_ptr(), *q_strides, k_data.data_ptr(), k_scale.data_ptr(), v_data.data_ptr(),
        v_scale.data_ptr(), *strides, block_table.data_ptr(), bt_stride if bt_rows > 1 else bt_cols,
        seq_lens.data_ptr(), out.data_ptr(), *out_strides, 0 if lse is None else lse.data_ptr(),
        0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(), _stream(dev),
        *form, kind, blocks, size, requests, query_len, max_seq_len, heads, kv, d, sm_scale))
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
    table's pages are not seen.  A row with no key has out 0 and lse -inf.
    Cached values that q's type does not hold (written from another type): V's
    count as +-6 * 2^13 (f16) or +-6 * 2^125 (bf16), K's as infinite."""
    lib = _library()
    if not isinstance(q, _torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    _need(idx, "idx", _torch.int32, _gpu(q, "q"), 2)
    rows, n_sel = idx.shape
    if rows != q.shape[0]:
        raise ValueError(f"idx must have one row per row of q ({q.shape[0]}), got {rows}")
    idx_stride, one = idx.stride()
    if n_sel > 1 and one != 1:
        raise ValueError("idx rows must be contiguous")
    if not isinstance(block_table, _torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [n_requests, max_blocks]")
    if not isinstance(k_data, _torch.Tensor) or k_data.dim() != 4:
        raise ValueError("k_data must be [n_blocks, block_size, n_kv_heads, head_dim/2]")
    if pool_size < 1:
        raise ValueError("pool_size must be >= 1")
    if n_sel == 0 and rows > 0:  # an empty selection has no address: one entry of -1 attends to as little
        idx = _torch.full((rows, 1), -1, dtype=_torch.int32, device=q.device)
        n_sel = idx_stride = 1
    return _attend(lib.indexer_mx4_attend_selected, q, k_data, k_scale, v_data, v_scale, block_table, seq_lens,
                   query_len, min(block_table.shape[1] * k_data.shape[1], MAX_KEYS), sm_scale, 1,
                   min(n_sel * pool_size, 2**31 - 1),
                   (idx.data_ptr(), idx_stride if rows > 1 else n_sel, n_sel, pool_size, 0, 0), out, lse, with_lse,
                   workspace)


def mx4_attend_window(q, k_data, k_scale, v_data, v_scale, block_table, seq_lens, query_len: int, max_seq_len: int,
                      sm_scale: float, window: int = 0, sinks: int = 0, out=None, lse=None, with_lse: bool = True,
                      workspace=None) -> Tuple:
    """Attention of each query row to its last `window` keys and the first
    `sinks` tokens (window 0: every key it sees): with v = seq_lens[r] - Q + 1
    + j, the keys s < min(v, max_seq_len) that have s >= v - window or
    s < sinks.  Other arguments and results as in mx4_attend_selected."""
    lib = _library()
    keys = max_seq_len if window == 0 else min(max_seq_len, window + sinks)
    return _attend(lib.indexer_mx4_attend_window, q, k_data, k_scale, v_data, v_scale, block_table, seq_lens, query_len,
                   max_seq_len, sm_scale, 0, max(0, min(keys, 2**31 - 1)),
                   (0, 0, 0, 0, window, sinks), out, lse, with_lse,
                   workspace)
