"""Rotary positions in fp64: rows x (B, h, S, d), a position per token, angles p * inv_freq[i]."""

from __future__ import annotations

import numpy as np


def rope_ref(x, inv_freq, positions, *, offset=0, interleaved=False, inverse=False, scale=1.0):
    """x (B, h, S, d) fp64 rotated pair by pair; positions (B, S). Pair i of the segment [offset, offset + 2 m)
    holds elements (i, m + i), or (2 i, 2 i + 1) when interleaved."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    m = len(inv_freq)
    for b in range(x.shape[0]):
        for t in range(x.shape[2]):
            for i in range(m):
                a = float(positions[b][t]) * float(inv_freq[i])
                c, s = scale * np.cos(a), scale * np.sin(-a if inverse else a)
                i0, i1 = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + m + i)
                out[b, :, t, i0] = x[b, :, t, i0] * c - x[b, :, t, i1] * s
                out[b, :, t, i1] = x[b, :, t, i1] * c + x[b, :, t, i0] * s
    return out
