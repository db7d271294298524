"""Head norms and rotation by position (``include/indexer_rope.h``).

What makes the rows that the indexer, the 4-bit cache and the attention take:
``norm_rope`` norms each head's row of queries and keys and rotates it by its
token's position, of one axis or of several.  Argument checks and marshalling
only, as in the rest of the binding.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Sequence, Tuple

from . import mx4 as _mx4

ROPE_EXPORTS = ("indexer_norm_rope",)
MAX_AXES = 4

# The argument structure of include/indexer_rope.h, member by member
NORM_ROPE = struct.Struct("=17q4Qq11i2f4x")

_lib = None
_torch = None


def _library():
    global _lib, _torch
    if _lib is None:
        lib = _mx4._library()
        lib.indexer_norm_rope.argtypes, lib.indexer_norm_rope.restype = [ctypes.c_char_p], ctypes.c_int
        _torch = _mx4._torch
        _lib = lib
    return _lib


@functools.lru_cache(maxsize=64)
def _axis_words(axes: Tuple[int, ...]) -> Tuple[int, int, int, int]:
    """Two bits a frequency, in four 64-bit words."""
    if len(axes) > 128 or not all(isinstance(i, int) and 0 <= i < MAX_AXES for i in axes):
        raise ValueError(f"axes must hold, for each of at most 128 frequencies, an axis in 0..{MAX_AXES - 1}")
    bits = sum(axis << (2 * i) for i, axis in enumerate(axes))
    return tuple((bits >> (64 * word)) & (2**64 - 1) for word in range(4))


def _weight(w, name, of, d, dev):
    """Checks a norm's weight; (address, 0: f32 or 1: of the rows' type)."""
    if w is None:
        return 0, 0
    if not isinstance(w, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = w.dtype
    if dtype is not _torch.float32 and dtype is not of:
        raise TypeError(f"{name} must be torch.float32 or {of}, got {dtype}")
    if w.get_device() != dev or w.dim() != 1:
        _mx4._need(w, name, dtype, dev, 1)
    if w.shape[0] != d or not w.is_contiguous():
        raise ValueError(f"{name} must hold one value per dimension ({d}), contiguous, got {list(w.shape)}")
    return w.data_ptr(), int(dtype is of)


def _out(given, like, name, dtype, dev, shape):
    """The output, a new one unless given, and its strides."""
    if given is None:
        return like.new_empty(shape), shape[1] * shape[2], shape[2]
    return (given, *_mx4._rows(given, name, dtype, dev, shape))


def norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
              axes: Optional[Sequence[int]] = None, interleaved: bool = False, rotary_scale: float = 1.0, q_out=None,
              k_out=None) -> Tuple:
    """Each head's RMS norm and the rotation by position, of queries and keys.

    q [n, q_heads, d] and k [n, k_heads, d] (or None), f16 or bf16, any token
    and head strides; positions i32 or i64 [n], or [n_axes, n] with `axes`
    naming the axis of each frequency (as images and video have them: time,
    height, width); inv_freq f32 [m], whose 2 m values of a row turn: value i
    with value i + m, or (interleaved) 2 i with 2 i + 1; the other values of a
    row pass.  A weight (f32 or of the rows' type, [d]) norms that tensor's
    rows by x / sqrt(mean(x^2) + eps) before; None does not.  The turned
    values are scaled by rotary_scale.  -> (q_out, k_out), new tensors unless
    given; an output may be its input.  No gradients."""
    lib = _library()
    torch = _torch
    dev = _mx4._gpu(q, "q")
    dtype = q.dtype
    kind = _mx4._types.get(dtype)
    if kind is None:
        raise TypeError(f"q must be torch.float16 or torch.bfloat16, got {dtype}")
    q_st, q_sh = _mx4._rows(q, "q", dtype, dev)
    n, heads, d = shape = q.shape
    q_out, q_ost, q_osh = _out(q_out, q, "q_out", dtype, dev, shape)
    k_ptr = k_out_ptr = k_heads = k_st = k_sh = k_ost = k_osh = 0
    if k is not None:
        k_st, k_sh = _mx4._rows(k, "k", dtype, dev)
        k_n, k_heads, k_d = k_shape = k.shape
        if k_n != n or k_d != d:
            raise ValueError(f"k must be [{n}, k_heads, {d}] as q, got {list(k_shape)}")
        k_out, k_ost, k_osh = _out(k_out, k, "k_out", dtype, dev, k_shape)
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    if not (isinstance(inv_freq, torch.Tensor) and inv_freq.dtype is torch.float32 and inv_freq.get_device() == dev
            and inv_freq.dim() == 1 and inv_freq.is_contiguous()):
        _mx4._need(inv_freq, "inv_freq", torch.float32, dev, 1)
        raise ValueError("inv_freq must be contiguous")
    freqs = inv_freq.shape[0]
    wide = isinstance(positions, torch.Tensor) and positions.dtype is torch.int64
    if not wide and not (isinstance(positions, torch.Tensor) and positions.dtype is torch.int32):
        raise TypeError("positions must be a torch.int32 or torch.int64 tensor")
    if positions.get_device() != dev or positions.dim() != (1 if axes is None else 2):
        _mx4._need(positions, "positions", positions.dtype, dev, 1 if axes is None else 2)
    if axes is None:
        n_axes, pos_stride, words = 1, 0, (0, 0, 0, 0)
    else:
        n_axes, pos_stride = positions.shape[0], positions.stride(0)
        axes = tuple(axes)
        if len(axes) != freqs:
            raise ValueError(f"axes must name an axis for each of the {freqs} frequencies, got {len(axes)}")
        words = _axis_words(axes)
    if positions.shape[-1] != n:
        raise ValueError(f"positions must have one entry per token ({n}), got {positions.shape[-1]}")
    if n > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must be contiguous along the tokens")
    q_w, q_kind = _weight(q_weight, "q_weight", dtype, d, dev)
    k_w, k_kind = _weight(k_weight, "k_weight", dtype, d, dev)
    if n == 0:  # nothing to do (and empty tensors have no address)
        return q_out, k_out
    _mx4._call(dev, lib.indexer_norm_rope, _mx4._pack(
        NORM_ROPE, q.data_ptr(), q_st, q_sh, k_ptr, k_st, k_sh, q_out.data_ptr(), q_ost, q_osh, k_out_ptr, k_ost, k_osh,
        q_w, k_w, positions.data_ptr(), pos_stride, inv_freq.data_ptr(), *words, _mx4._stream(dev), kind, n, heads,
        k_heads, d, freqs, n_axes, int(bool(interleaved)), int(wide), q_kind, k_kind, eps, rotary_scale))
    return q_out, k_out
