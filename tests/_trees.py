"""Drafted trees and windowed caches shared by the tree operators' tests."""
import numpy as np

import oracle
from tests._serving import PagedCase, f64


def random_parents(rng, B, N, deepest=None, shape="random"):
    """[B, N] int32 parents: random trees, or chains, stars (every node a child of the root) or forests."""
    out = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, N):
            if shape == "chain":
                out[b, i] = i - 1
            elif shape == "star":
                out[b, i] = 0
            elif shape == "forest":
                out[b, i] = rng.integers(-1, i)
            else:
                p = int(rng.integers(0, i))
                while deepest is not None and oracle.depths(out[b, :i])[p] >= deepest:
                    p = int(rng.integers(0, i))
                out[b, i] = p
    return out


class TreeCase(PagedCase):
    """A paged cache whose requests' last tokens are the nodes of a tree."""

    def __init__(self, *args, parents, window=0, sinks=0, **kw):
        super().__init__(*args, **kw)
        self.parents, self.window, self.sinks = np.asarray(parents, np.int32), window, sinks

    def run(self, ds, lengths=None, causal=True, workspace=None, out=None):
        import torch
        B, N, Hq, _ = self.q.shape
        lse = torch.full((B, N, Hq), 7.0, device="cuda")
        dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()
        out = ds.dspark_tree_attention(self.q, self.k, self.v, dev(self.table), dev(self.kv_len), dev(self.parents), self.scale,
                                       lengths=dev(lengths), window=self.window, sinks=self.sinks, lse=lse, workspace=workspace,
                                       out=out)
        return out, lse

    def sees(self, b, i, lengths, causal):
        L, n = int(self.kv_len[b]), self.N if lengths is None else int(lengths[b])
        return oracle.tree_row_sees(L, n, i, self.parents[b].tolist(), self.window, self.sinks) if i < n and L >= n else []

    def row(self, b, i, h, lengths=None, causal=True):
        j = np.array(self.sees(b, i, lengths, causal), dtype=int)
        pages, offs = self.table[b, j // self.page], j % self.page
        hk, D = h // self.group, self.q.shape[-1]
        K, V = f64(self.k[pages, hk, offs]), f64(self.v[pages, hk, offs])
        return oracle.attend_row(f64(self.q[b, i, h]), K.reshape(-1, D), V.reshape(-1, D), self.scale)


class WindowCase(TreeCase):
    """A paged cache that is seen through a window and sinks."""

    def __init__(self, *args, window, sinks, **kw):
        super().__init__(*args, parents=np.zeros((0,)), window=window, sinks=sinks, **kw)

    def run(self, ds, lengths=None, causal=True, workspace=None, out=None):
        import torch
        B, N, Hq, _ = self.q.shape
        lse = torch.full((B, N, Hq), 7.0, device="cuda")
        dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()
        out = ds.dspark_window_attention(self.q, self.k, self.v, dev(self.table), dev(self.kv_len), self.window, self.sinks,
                                         self.scale, lengths=dev(lengths), causal=causal, lse=lse, workspace=workspace, out=out)
        return out, lse

    def sees(self, b, i, lengths, causal):
        L, n = int(self.kv_len[b]), self.N if lengths is None else int(lengths[b])
        return oracle.window_row_sees(L, n, i, self.window, self.sinks, causal) if i < n else []
