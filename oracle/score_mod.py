"""Attention with modified scores (a cap by tanh, a distance bias, a key range per row) and its gradients, in fp64."""

from __future__ import annotations

import numpy as np


def _rows(q, k, b, a, r, at, n, scale, softcap, slopes, seen):
    """Probabilities, lse and the cap's derivative of head a's rows over the first n keys."""
    z = scale * (q[b, a] @ k[b, a // r, :n].T)
    slope_of_cap = np.ones_like(z)
    if softcap:
        t = np.tanh(z / softcap)
        z, slope_of_cap = softcap * t, 1.0 - t * t
    if slopes is not None:
        z = z - slopes[a] * np.abs(at[:, None] - np.arange(n)[None, :])
    z = np.where(seen, z, -np.inf)
    top = z.max(1, initial=-np.inf)
    e = np.exp(z - np.where(np.isfinite(top), top, 0.0)[:, None])
    l = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, top + np.log(np.where(l > 0, l, 1.0)), -np.inf)
    return e / np.where(l > 0, l, 1.0)[:, None], lse, slope_of_cap


def modified_attention_ref(q, k, v, *, q_start=None, kv_len=None, scale=None, causal=True, window=0, softcap=0.0,
                           slopes=None, key_range=None, d_o=None):
    """(o, lse, weighted |v|) of q (B, h_q, S, d) over k, v (B, h_kv, T, d), and with d_o also (dq, dk, dv). Keys at and
    past kv_len are not read. Rows that see no key: zeros, lse -inf."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, h_q, S, d = q.shape
    h_kv, T = k.shape[1:3]
    r = h_q // h_kv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, mag, lse = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:3])
    dq, dk, dv = np.zeros_like(q), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        n = T if kv_len is None else int(kv_len[b])
        at = (0 if q_start is None else int(q_start[b])) + np.arange(S)
        key = np.arange(n)[None, :]
        seen = np.ones((S, n), bool)
        if causal:
            seen &= key <= at[:, None]
            if window:
                seen &= key > at[:, None] - window
        if key_range is not None:
            seen &= (key >= key_range[b, :, :1]) & (key < key_range[b, :, 1:])
        for a in range(h_q):
            g = a // r
            p, lse[b, a], slope_of_cap = _rows(q, k, b, a, r, at, n, scale, softcap, slopes, seen)
            o[b, a], mag[b, a] = p @ v[b, g, :n], p @ np.abs(v[b, g, :n])
            if d_o is not None:
                up = np.asarray(d_o[b, a], np.float64)
                ds = p * (up @ v[b, g, :n].T - (up * o[b, a]).sum(1, keepdims=True)) * slope_of_cap * scale
                dq[b, a] = ds @ k[b, g, :n]
                dk[b, g, :n] += ds.T @ q[b, a]
                dv[b, g, :n] += p.T @ up
    return (o, lse, mag) if d_o is None else (o, lse, mag, dq, dk, dv)
