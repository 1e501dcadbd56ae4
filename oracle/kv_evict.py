"""Which cached keys an eviction keeps, from the rule alone."""

from __future__ import annotations

import numpy as np


def kv_evict_ref(weights, kv_len, budget, *, sink=0, recent=0):
    """kept (B, h_kv, budget) ascending rows (-1 past the new length) and new_len (B): the first ``sink`` and the last
    ``recent`` of n rows, and the heaviest of the others, ties to the lower row, NaN below every number."""
    B, h_kv, _ = weights.shape
    kept = np.full((B, h_kv, budget), -1, np.int32)
    for b in range(B):
        n = int(kv_len[b])
        for g in range(h_kv):
            if n <= budget:
                keep = list(range(n))
            else:
                w = weights[b, g]
                order = sorted(range(sink, n - recent), key=lambda j: (np.isnan(w[j]), -w[j] if w[j] == w[j] else 0, j))
                keep = sorted([*range(sink), *order[:budget - sink - recent], *range(n - recent, n)])
            kept[b, g, :len(keep)] = keep
    return kept, np.minimum(np.asarray(kv_len, np.int32), budget)
