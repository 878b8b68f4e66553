"""Position rotation, per-head norm and the paged cache's writes (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Source: "DSpark implementation and evaluation" §4: the context-KV precompute normalises the keys
per head (RMS), rotates them by position and writes keys and values to the cache.  A rotation turns
each pair (a, b) of a head's first `rot` values by the token's angle: (a cos - b sin, b cos + a sin).
"""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, cos, sin, interleaved=False):
    """x [T, H, D] with cos and sin [T, rot / 2]: pairs (x[i], x[i + rot/2]), or (x[2i], x[2i + 1])."""
    x = np.array(x, dtype=np.float64)
    half = cos.shape[1]
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[:, :, ia].copy(), x[:, :, ib].copy()
        c, s = cos[:, i, None].astype(np.float64), sin[:, i, None].astype(np.float64)
        x[:, :, ia] = a * c - b * s
        x[:, :, ib] = b * c + a * s
    return x


def kv_append(q, k, v, positions, slots, cos_sin, k_cache, v_cache, interleaved=False, q_norm=None, k_norm=None,
              eps=1e-6):
    """Returns (q_out, k_cache, v_cache) in float64; a token with slot -1 leaves the caches alone."""
    half = cos_sin.shape[1] // 2
    cs = np.asarray(cos_sin)[np.asarray(positions)]
    cos, sin = cs[:, :half], cs[:, half:]
    kr = rotate(k if k_norm is None else rms_norm(k, k_norm, eps), cos, sin, interleaved)
    qr = None if q is None else rotate(q if q_norm is None else rms_norm(q, q_norm, eps), cos, sin, interleaved)
    K, V = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    page = K.shape[2]
    for t, slot in enumerate(slots):
        if slot >= 0:
            K[slot // page, :, slot % page] = kr[t]
            V[slot // page, :, slot % page] = np.asarray(v[t], dtype=np.float64)
    return qr, K, V
