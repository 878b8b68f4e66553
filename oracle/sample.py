"""Truncated sampling: temperature, top-k, min-p, top-p and an inverse-CDF draw (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

The truncations are the usual ones of serving requests; "Speculative decoding: from zero to DSpark"
§2 verifies whatever distributions it is given, so a truncated target is verified by truncating
p_t.  The masses are integers as in the residual draw of verification (q = floor(w * 2^40)), so the
kept set and the token are functions of the weights alone and of no order of summation; they are
computed here with Python integers, entry by entry.
"""
from __future__ import annotations

import math

import numpy as np

MASS = 2 ** 40
FRAC = 2 ** 24


def weights(x, temperature):
    """w_v = exp((x_v - m) / T) of one row in float64 (NaN, +-infinity: 0); T = 0: one at every largest entry."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    if not ok.any():
        return np.zeros(x.shape)
    m = x[ok].max()
    if temperature == 0:
        return np.where(ok & (x == m), 1.0, 0.0)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(ok, np.exp(np.where(ok, x - m, -math.inf) / temperature), 0.0)


def sample_row(x, w, temperature, top_k, top_p, min_p, u):
    """One row from its logits x (for the order) and fp32 weights w; returns (token, kept ids, masses, total).

    kept ids are in the order of the entries (logit descending, id ascending)."""
    x = np.asarray(x, dtype=np.float64)
    ids = [int(v) for v in sorted((v for v in range(len(x)) if np.isfinite(x[v])), key=lambda v: (-x[v], v))]
    if not ids:
        return 0, [], [], 0
    k = 1 if temperature == 0 else (top_k if top_k > 0 else len(x))
    ids = [v for v in ids[:k] if np.float32(w[v]) >= np.float32(min_p)]
    mass = [int(math.floor(float(w[v]) * MASS)) for v in ids]
    need = sum(mass) * int(math.floor(float(np.float32(top_p)) * FRAC)) // FRAC
    before, kept, left = 0, [], []
    for n, (v, q) in enumerate(zip(ids, mass)):
        if n > 0 and before >= need:
            break
        kept.append(v)
        left.append(q)
        before += q
    total = sum(left)
    target = total * int(math.floor(float(np.float32(u)) * FRAC)) // FRAC
    by_id = sorted(zip(kept, left))
    run = 0
    for v, q in by_id:
        run += q
        if run > target:
            return v, kept, left, total
    return by_id[-1][0], kept, left, total


def truncated_distribution(x, temperature, top_k, top_p, min_p):
    """The kept entries' distribution in float64 arithmetic throughout, for one row."""
    w = weights(x, temperature)
    _, kept, left, total = sample_row(x, w, temperature, top_k, top_p, min_p, 0.0)
    p = np.zeros(len(x))
    for v, q in zip(kept, left):
        p[v] = q / total
    return p
