"""Inputs and derived tolerances shared by the serving operators' GPU tests."""
import math

import numpy as np

import oracle

# half the spacing of a type at 1 (round-to-nearest's relative error): 8 and 11 significant bits
ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def half_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def f64(t):
    return t.double().cpu().numpy()


def attention_tolerance(ref_out, spread, size, dtype, keys, vmax):
    """Bound on |out - ref| per value.

    out is rounded once to the type (ULP |out|).  Each weight is rounded to the type before its
    product (ULP of it, so at most ULP * spread in the sum, spread = sum p |v|); the weights'
    own sum may or may not hold those roundings: another ULP * |out| <= ULP * spread.  fp32
    scores are off by at most (D + 2) 2^-24 `size` < 2^-16 size, which moves a weight by that
    factor in numerator and sum.  2^-18 covers the exponential (2 ulp) and fp32 sums in tiles.  fp16
    weights below 2^-14 of the row's largest are rounded to 2^-25 of it instead: keys * 2^-25
    * vmax at most, doubled for a reference up to 2^8 below the largest (they are then larger).
    """
    u = ULP[dtype]
    tol = u * np.abs(ref_out) + 2 * u * spread + 2 * (size[..., None] * 2.0 ** -16 + 2.0 ** -18) * spread
    if dtype == "f16":
        tol = tol + 2 * keys * 2.0 ** -25 * vmax + 2.0 ** -25
    return tol * 1.01 + 1e-30


def lse_tolerance(lse, size):
    """Scores as above, the sum's own rounding and the logarithm's (and that of the result in fp32)."""
    return size * 2.0 ** -16 + 2.0 ** -17 + np.abs(np.where(np.isfinite(lse), lse, 0.0)) * 2.0 ** -22


def check_attention(got_out, got_lse, ref, dtype, keys, vmax):
    out, lse, spread, size = ref
    g = f64(got_out)
    assert g.shape == out.shape
    nan = np.isnan(out)
    np.testing.assert_array_equal(np.isnan(g), nan)
    err = np.abs(np.where(nan, 0.0, g - out))
    tol = np.where(nan, 0.0, attention_tolerance(out, spread, size, dtype, keys, vmax))
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"out off at {worst}: {g[worst]} for {out[worst]}, tolerance {tol[worst]}"
    if got_lse is not None:
        gl = f64(got_lse)
        empty = lse == -math.inf
        np.testing.assert_array_equal(gl == -math.inf, empty)
        err = np.abs(np.where(empty, 0.0, gl - np.where(empty, 0.0, lse)))
        assert (err <= lse_tolerance(lse, size)).all(), f"lse off by {err.max()}"


class PagedCase:
    """A paged cache with its tokens in shuffled pages, and NaN in every slot that holds no token."""

    def __init__(self, B, N, Hq, Hkv, D, page, kv_len, dtype="bf16", seed=0, spare=3, gain=1.0, extra_width=2):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.scale = dtype, D ** -0.5
        dt = half_dtype(dtype)
        rng = np.random.default_rng(seed)
        need = [-(-L // page) for L in kv_len]
        P = sum(need) + spare
        order = rng.permutation(P)
        width = max(need) + extra_width
        table = np.full((B, width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        shape = (P, Hkv, page, D)
        self.k = torch.randn(shape, generator=g, device="cuda").to(dt)
        self.v = torch.randn(shape, generator=g, device="cuda").to(dt)
        hold = np.zeros((P, page), bool)
        for b, L in enumerate(kv_len):
            for p in range(need[b]):
                hold[table[b, p], :max(0, min(page, L - p * page))] = True
        hold = torch.from_numpy(hold).cuda()[:, None, :, None]
        self.k = torch.where(hold, self.k, math.nan)
        self.v = torch.where(hold, self.v, math.nan)
        self.q = (torch.randn(B, N, Hq, D, generator=g, device="cuda") * gain).to(dt)
        self.table, self.kv_len = table, np.asarray(kv_len, np.int32)
        self.page, self.N, self.group = page, N, Hq // Hkv

    def run(self, ds, lengths=None, causal=True, workspace=None, out=None):
        import torch
        B, N, Hq, _ = self.q.shape
        lse = torch.full((B, N, Hq), 7.0, device="cuda")
        ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        out = ds.dspark_paged_attention(self.q, self.k, self.v, torch.from_numpy(self.table).cuda(),
                                        torch.from_numpy(self.kv_len).cuda(), self.scale, lengths=ln, causal=causal,
                                        lse=lse, workspace=workspace, out=out)
        return out, lse

    def row(self, b, i, h, lengths=None, causal=True):
        """The oracle's (out, lse, spread, size) of one row."""
        L, n = int(self.kv_len[b]), self.N if lengths is None else int(lengths[b])
        limit = 0 if i >= n else max(0, L - n + i + 1) if causal else L
        j = np.arange(limit)
        pages, offs = self.table[b, j // self.page], j % self.page
        hk = h // self.group
        K, V = f64(self.k[pages, hk, offs]), f64(self.v[pages, hk, offs])
        D = self.q.shape[-1]
        return oracle.attend_row(f64(self.q[b, i, h]), K.reshape(limit, D), V.reshape(limit, D), self.scale)

    def check(self, ds, lengths=None, causal=True, rows=None, seed=0, **kw):
        out, lse = self.run(ds, lengths, causal, **kw)
        B, N, Hq, _ = self.q.shape
        every = [(b, i, h) for b in range(B) for i in range(N) for h in range(Hq)]
        if rows is not None and rows < len(every):
            pick = np.random.default_rng(seed).choice(len(every), rows, replace=False)
            every = [every[p] for p in pick]
        ref = [np.array(x) for x in zip(*(self.row(b, i, h, lengths, causal) for b, i, h in every))]
        at = tuple(np.array(x) for x in zip(*every))
        import torch
        at = tuple(torch.from_numpy(x).cuda() for x in at)
        check_attention(out[at], lse[at], ref, self.dtype, int(self.kv_len.max()) if len(self.kv_len) else 0, 6.0)
        return out, lse
