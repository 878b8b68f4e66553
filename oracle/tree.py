"""Trees of drafted tokens and windows: what a row sees, which path is accepted, how the cache follows (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

"Speculative decoding: from zero to DSpark" §2 scores one drafted block in one pass and keeps the longest accepted
prefix; with several candidates per position the block is a tree, and what is kept is a path from its root.  The
target's own token decides at every node, so the tokens put out have the target's law whatever the tree holds.
Every function is a plain loop.
"""
from __future__ import annotations

import numpy as np

from .sample import sample_row


def depths(parents):
    """Number of ancestors of every node of one tree."""
    out = []
    for p in parents:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def window_row_sees(L, n, i, window, sinks, causal=True):
    """Cached tokens, in order, that new token i of n sees (L cached ones, its own among them)."""
    p = L - n + i
    return [j for j in range(L) if (j <= p or not causal) and (j < sinks or j > p - window)]


def tree_row_sees(L, n, i, parents, window=0, sinks=0):
    """Cached tokens, in order, that node i of a tree of n sees."""
    base = L - n
    p = base + depths(parents[:n])[i]
    sees = {j for j in range(base) if window == 0 or j < sinks or j > p - window}
    at = i
    while at >= 0:
        sees.add(base + at)
        at = parents[at]
    return sorted(sees)


def verify_tree(next_token, parents, tokens, n):
    """One request: next_token(node) gives the target's token behind a node.  Returns (tokens out, path)."""
    if n == 0:
        return [], []
    out, path = [], [0]
    while True:
        y = next_token(path[-1])
        out.append(y)
        child = [i for i in range(1, n) if parents[i] == path[-1] and tokens[i] == y]
        if not child:
            return out, path
        path.append(child[0])


def tree_token(x, w, temperature, u):
    """The target's token of one row (logits x, fp32 weights w): the draw without top-k, top-p and min-p."""
    return sample_row(x, w, temperature, 0, 1.0, 0.0, u)[0]


def compact(cache, table, kv_len, n, path, accepted):
    """cache [layers, P, Hkv, page, D] of one request; returns (new cache, new length)."""
    cache = np.array(cache)
    if n == 0:
        return cache, kv_len
    page, base = cache.shape[3], kv_len - n
    old = cache.copy()
    for i in range(accepted + 1):
        a, z = base + path[i], base + i
        cache[:, table[z // page], :, z % page] = old[:, table[a // page], :, a % page]
    return cache, base + accepted + 1


def copy_pages(cache, src, dst, used=None):
    """cache [layers, P, Hkv, page, D]; the first used[m] tokens of page dst[m] become those of page src[m]."""
    old, cache = np.array(cache), np.array(cache)
    for m, (a, z) in enumerate(zip(src, dst)):
        n = cache.shape[3] if used is None else used[m]
        cache[:, z, :, :n] = old[:, a, :, :n]
    return cache
