"""Attention weight of every cached key in fp64, from given lse values."""

from __future__ import annotations

import numpy as np


def kv_weights_ref(q, k, lse, *, q_start=None, kv_len=None, scale=None, causal=True, window=0):
    """(B, h_kv, T): sum over the group's heads and rows that see key j of exp(scale q.k - lse). q (B, h_q, S, d),
    k (B, h_kv, T, d), lse (B, h_q, S); q_start None: the rows are the last S cached positions; rows with lse
    -inf or NaN add nothing."""
    q, k, lse = (np.asarray(x, np.float64) for x in (q, k, lse))
    B, h_q, S, d = q.shape
    h_kv, T = k.shape[1:3]
    r = h_q // h_kv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    w = np.zeros((B, h_kv, T))
    for b in range(B):
        n = T if kv_len is None else int(kv_len[b])
        start = n - S if q_start is None else int(q_start[b])
        at = start + np.arange(S)[:, None]
        key = np.arange(n)[None, :]
        seen = np.ones((S, n), bool)
        if causal:
            seen &= key <= at
            if window:
                seen &= key > at - window
        for a in range(h_q):
            rows = np.isfinite(lse[b, a])
            s = scale * (q[b, a][rows] @ k[b, a // r, :n].T) - lse[b, a][rows][:, None]
            w[b, a // r, :n] += np.where(seen[rows], np.exp(np.where(seen[rows], s, 0.0)), 0.0).sum(0)
    return w
