"""Plain 64-bit forms of the 4-bit cache and the attention over it, in NumPy.

Test infrastructure, like the rest of this package: written from the
definitions in include/indexer_mx4.h, one row at a time, sharing no code with
the HIP path.  bf16 values are passed as float32 arrays that hold them exactly.
"""
from __future__ import annotations

import math

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
RANGE = {"f16": (-23, 13), "bf16": (-126, 125)}


def exponent(amax: float, kind: str) -> int:
    """The least e in the type's range with amax < 7 * 2^e, or the range's end."""
    lo, hi = RANGE[kind]
    for e in range(lo, hi):
        if amax < math.ldexp(7.0, e):
            return e
    return hi


def code(y: float) -> int:
    """The 4-bit code nearest y: ties to the even code, at most 6 in magnitude."""
    a = abs(y)
    best = min(range(8), key=lambda i: (abs(a - MAGNITUDES[i]), i % 2)) if a < 6.0 else 7
    return best + (8 if math.copysign(1.0, y) < 0 else 0)


def quantise(x: np.ndarray, kind: str):
    """Rows [..., d] -> (codes packed [..., d/2] u8, scales [..., d/32] u8)."""
    d = x.shape[-1]
    blocks = x.astype(np.float64).reshape(-1, 32)
    codes = np.zeros(blocks.shape, dtype=np.uint8)
    scales = np.empty(len(blocks), dtype=np.uint8)
    for i, b in enumerate(blocks):
        if not np.all(np.isfinite(b)):
            scales[i] = 255
            continue
        e = exponent(float(np.max(np.abs(b))), kind)
        scales[i] = e + 127
        codes[i] = [code(math.ldexp(float(v), -e)) for v in b]
    flat = codes.reshape(-1, 2)
    return ((flat[:, 0] | (flat[:, 1] << 4)).reshape(x.shape[:-1] + (d // 2,)),
            scales.reshape(x.shape[:-1] + (d // 32,)))


def values(data: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """f64 values [..., d] of packed codes [..., d/2] and scales [..., d/32]."""
    codes = np.stack([data & 15, data >> 4], -1).reshape(data.shape[:-1] + (-1, 32))
    v = np.where(codes >= 8, -1.0, 1.0) * MAGNITUDES[codes & 7]
    with np.errstate(invalid="ignore"):
        f = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
        return (v * f[..., None]).reshape(data.shape[:-1] + (-1,))


def positions_selected(idx_row, pool: int, seen: int):
    """The positions a selection names, of those below `seen`, in order."""
    return [int(i) * pool + u for i in idx_row if i >= 0 for u in range(pool) if int(i) * pool + u < seen]


def positions_window(v: int, seen: int, window: int, sinks: int):
    return [p for p in range(max(seen, 0)) if window == 0 or p >= v - window or p < sinks]


def attend_rows(q, rows_k, rows_v, block_table, seq_lens, query_len, max_seq_len, sm_scale, positions):
    """The attention of every row, in f64.

    q [R*Q, H, d]; rows_k, rows_v [n_blocks, block_size, KV, d]; positions(t,
    v, seen) the positions row t attends to.  Returns out, lse, and for the
    tests' error bounds: weight * |V| summed (like out), the largest
    sm_scale * |q| . |k| and the largest |z| of each row and head, the number
    of keys, and sum |V| (like out)."""
    q = q.astype(np.float64)
    rows, H, d = q.shape
    n_blocks, bs, kv, _ = rows_k.shape
    g = H // kv
    out, spread, plain = (np.zeros((rows, H, d)) for _ in range(3))
    lse = np.full((rows, H), -np.inf)
    reach, top = np.zeros((rows, H)), np.zeros((rows, H))
    count = np.zeros(rows, dtype=np.int64)
    for t in range(rows):
        r, j = divmod(t, query_len)
        v = int(seq_lens[r]) - query_len + 1 + j
        pos = np.array(positions(t, v, min(v, max_seq_len)), dtype=np.int64)
        if pos.size:
            page = block_table[r, pos // bs].astype(np.int64)
            keep = (page >= 0) & (page < n_blocks)
            pos, page = pos[keep], page[keep]
        count[t] = pos.size
        if not pos.size:
            continue
        k, val = rows_k[page, pos % bs], rows_v[page, pos % bs]
        for h in range(H):
            z = sm_scale * (k[:, h // g] @ q[t, h])
            m = np.max(z)
            w = np.exp(z - m)
            lse[t, h] = m + math.log(np.sum(w)) if not np.isnan(m) else np.nan
            w = w / np.sum(w)
            with np.errstate(invalid="ignore"):
                out[t, h] = w @ val[:, h // g]
                spread[t, h] = w @ np.abs(val[:, h // g])
                plain[t, h] = np.sum(np.abs(val[:, h // g]), 0)
                reach[t, h] = sm_scale * np.max(np.abs(k[:, h // g]) @ np.abs(q[t, h]))
                top[t, h] = np.max(np.abs(z))
    return out, lse, {"spread": spread, "reach": reach, "top": top, "count": count, "plain": plain}
