"""Attention over a paged cache and within packed prompts (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Sources: "Speculative decoding: from zero to DSpark" §2 (the target scores the drafted block in
one pass) and "DSpark implementation and evaluation" §4 (the draft backbone's block of N query
tokens, non-causal over the context KV).  The pages name attention without spelling it out; it is
softmax(scale * q k^T) v with heads in groups, over the tokens a row may see.  A row that sees
nothing gives 0 and log-sum-exp -infinity.

Every function is a plain loop over rows in float64; a row only touches the keys and values it
sees.  Beside the result each returns, per row, sum_j p_j |v_j| and the largest
scale * sum_d |q_d k_d|, which bound what rounding can do to the row.
"""
from __future__ import annotations

import math

import numpy as np


def attend_row(q, K, V, scale):
    """One row: q [D], K and V [n, D]; returns (out [D], lse, spread [D], size)."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    if K.shape[0] == 0:
        return np.zeros(V.shape[1]), -math.inf, np.zeros(V.shape[1]), 0.0
    s = (K @ q) * scale
    size = float(np.max(np.abs(K) @ np.abs(q)) * abs(scale))
    m = s.max()
    if m == -math.inf:                       # every score is -infinity: no weight anywhere
        return np.zeros(V.shape[1]), -math.inf, np.zeros(V.shape[1]), size
    w = np.exp(s - m)
    total = w.sum()
    return (w @ V) / total, m + math.log(total), (w @ np.abs(V)) / total, size


def paged_attention(q, k_cache, v_cache, block_table, kv_len, scale, lengths=None, causal=True):
    """q [B, N, Hq, D], caches [P, Hkv, page, D]; returns (out, lse, spread, size) with leading [B, N, Hq]."""
    q, k_cache, v_cache = (np.asarray(x) for x in (q, k_cache, v_cache))
    B, N, Hq, D = q.shape
    _, Hkv, page, _ = k_cache.shape
    out, spread = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    lse, size = np.full((B, N, Hq), -math.inf), np.zeros((B, N, Hq))
    for b in range(B):
        L, n = int(kv_len[b]), N if lengths is None else int(lengths[b])
        for i in range(n):
            limit = max(0, L - n + i + 1) if causal else L
            where = [(int(block_table[b][j // page]), j % page) for j in range(limit)]
            pages, offs = [w[0] for w in where], [w[1] for w in where]
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                out[b, i, h], lse[b, i, h], spread[b, i, h], size[b, i, h] = attend_row(
                    q[b, i, h], k_cache[pages, hk, offs].reshape(-1, D), v_cache[pages, hk, offs].reshape(-1, D), scale)
    return out, lse, spread, size


def prompt_attention(q, k, v, cu_seqlens, scale, causal=True):
    """q [T, Hq, D], k and v [T, Hkv, D]; returns (out, lse, spread, size) with leading [T, Hq]."""
    q, k, v = (np.asarray(x) for x in (q, k, v))
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    out, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, size = np.full((T, Hq), -math.inf), np.zeros((T, Hq))
    for a, z in zip(cu_seqlens[:-1], cu_seqlens[1:]):
        for t in range(int(a), int(z)):
            end = t + 1 if causal else int(z)
            for h in range(Hq):
                out[t, h], lse[t, h], spread[t, h], size[t, h] = attend_row(
                    q[t, h], k[int(a):end, h // group], v[int(a):end, h // group], scale)
    return out, lse, spread, size
