"""The plain 64-bit form of the head norm and rotation, in NumPy.

Test infrastructure, written from the definition in include/indexer_rope.h,
sharing no code with the HIP path.  bf16 values are passed as float64 arrays
that hold them exactly.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, weight, positions, inv_freq, axes, eps, interleaved, rotary_scale):
    """x [n, heads, d] f64, weight [d] or None, positions [n_axes, n], inv_freq
    [m], axes [m].  Returns the rows, the magnitudes each value is a sum of
    (for error bounds), and the angles [n, m]."""
    x = x.astype(np.float64)
    m = len(inv_freq)
    with np.errstate(all="ignore"):
        if weight is not None:
            x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * weight
        angle = np.array([[float(positions[axes[i], t]) * float(inv_freq[i]) for i in range(m)]
                          for t in range(x.shape[0])]).reshape(x.shape[0], m)
        out, reach = x.copy(), np.abs(x)
        for i in range(m):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
            c, s = np.cos(angle[:, i])[:, None], np.sin(angle[:, i])[:, None]
            out[..., a] = rotary_scale * (x[..., a] * c - x[..., b] * s)
            out[..., b] = rotary_scale * (x[..., b] * c + x[..., a] * s)
            reach[..., a] = reach[..., b] = abs(rotary_scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, reach, angle
