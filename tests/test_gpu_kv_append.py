"""GPU parity: appending rotated keys and values to a paged cache, against the 64-bit oracle."""
import numpy as np
import pytest

import oracle
from tests._serving import ULP, f64, half_dtype

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, Hq, Hkv, D, rot, page, pages, dtype, seed, pad=0, positions=500):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, dt = dtype, half_dtype(dtype)
        rows = torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g, device="cuda").to(dt)
        q, k, v, _ = rows.split([Hq * D, Hkv * D, Hkv * D, 8], dim=1)
        self.q = q.view(T, Hq, D) if Hq else None
        self.k, self.v = k.view(T, Hkv, D), v.view(T, Hkv, D)
        slots = rng.permutation(pages * page)[:T].astype(np.int32)
        slots[rng.permutation(T)[:pad]] = -1
        self.slots = slots
        self.positions = rng.integers(0, positions, T).astype(np.int32)
        ang = np.arange(positions)[:, None] * 100.0 ** -(np.arange(rot // 2) / max(1, rot // 2))
        self.cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)
        self.k_cache = torch.randn(pages, Hkv, page, D, generator=g, device="cuda").to(dt)
        self.v_cache = torch.randn(pages, Hkv, page, D, generator=g, device="cuda").to(dt)
        self.q_norm = torch.randn(D, generator=g, device="cuda") * 0.2 + 1
        self.k_norm = torch.randn(D, generator=g, device="cuda") * 0.2 + 1

    def call(self, ds, interleaved=False, norm=False, **kw):
        import torch
        K, V = self.k_cache.clone(), self.v_cache.clone()
        q = ds.dspark_kv_append(self.q, self.k, self.v, torch.from_numpy(self.positions).cuda(),
                                torch.from_numpy(self.slots).cuda(), torch.from_numpy(self.cos_sin).cuda(), K, V,
                                interleaved=interleaved, q_norm=self.q_norm if norm else None,
                                k_norm=self.k_norm if norm else None, **kw)
        return q, K, V

    def check(self, ds, interleaved=False, norm=False, **kw):
        got = self.call(ds, interleaved, norm, **kw)
        ref = oracle.kv_append(None if self.q is None else f64(self.q), f64(self.k), f64(self.v), self.positions,
                               self.slots, self.cos_sin, f64(self.k_cache), f64(self.v_cache), interleaved,
                               f64(self.q_norm) if norm else None, f64(self.k_norm) if norm else None)
        # One rounding to the type (fp16 below 2^-14: to 2^-25), plus fp32 ahead of it: the sum of
        # squares and root (D 2^-24 < 2^-15 relative), three roundings of products and a sum whose
        # terms are at most sqrt(2) times the pair's length; |values| < 8 here.
        for x, y in zip(got, ref):
            if x is None:
                continue
            tol = ULP[self.dtype] * np.abs(y) * 1.01 + 8 * 1.5 * 2.0 ** -15 + 2.0 ** -25
            np.testing.assert_array_less(np.abs(f64(x) - y), tol)
        import torch
        assert torch.equal(got[2], _scatter(self.v_cache, self.v, self.slots))        # values are copied
        held = np.zeros(self.k_cache.shape[0] * self.k_cache.shape[2], bool)
        held[self.slots[self.slots >= 0]] = True
        other = torch.from_numpy(~held.reshape(self.k_cache.shape[0], 1, -1, 1)).cuda().expand_as(self.k_cache)
        assert torch.equal(got[1][other], self.k_cache[other])                        # the rest is left alone
        return got


def _scatter(cache, new, slots):
    import torch
    out = cache.clone()
    page = cache.shape[2]
    at = torch.from_numpy(slots.astype(np.int64)).cuda()
    ok = at >= 0
    out[at[ok] // page, :, at[ok] % page] = new[ok]
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (16, 16), (80, 32), (96, 0), (256, 256), (512, 496),
                                   (48, 48)])
def test_head_sizes_rotations_and_types(cuda_lib, dtype, interleaved, D, rot):
    case = Case(37, 5, 2, D, rot, 16, 6, dtype, seed=D + rot, pad=4)
    case.check(cuda_lib, interleaved, norm=False)
    case.check(cuda_lib, interleaved, norm=True)


@pytest.mark.parametrize("T,Hq,Hkv,page", [(1, 1, 1, 1), (1, 32, 8, 16), (2, 0, 3, 7), (1000, 32, 8, 16), (333, 71, 1, 48),
                                           (3000, 16, 16, 64)])
def test_sizes(cuda_lib, T, Hq, Hkv, page):
    case = Case(T, Hq, Hkv, 64, 64, page, T // page + 2, "bf16", seed=T, pad=T // 10)
    case.check(cuda_lib, norm=T % 2 == 0)


@pytest.mark.parametrize("T,D,rot,interleaved", [(4501, 80, 32, False), (4501, 128, 64, True), (1103, 512, 496, True),
                                                 (35003, 16, 16, False), (9001, 48, 48, True)])
def test_many_tokens(cuda_lib, T, D, rot, interleaved):
    # several rows to a lane, more of them than the last lanes' rows (9 heads)
    case = Case(T, 5, 2, D, rot, 16, T // 16 + 2, "f16", seed=T + D, pad=T // 7)
    case.check(cuda_lib, interleaved, norm=False)
    case.check(cuda_lib, interleaved, norm=True)


def test_in_place_queries_streams_and_graphs(cuda_lib):
    import torch
    case = Case(50, 4, 2, 128, 128, 16, 8, "bf16", seed=3)
    want = case.call(cuda_lib)
    q = case.q.contiguous()
    case.q = q.clone()
    got = case.call(cuda_lib, q_out=case.q)
    assert got[0].data_ptr() == case.q.data_ptr() and torch.equal(got[0], want[0])
    case.q = q
    pos, slots = torch.from_numpy(case.positions).cuda(), torch.from_numpy(case.slots).cuda()
    cs, K, V = torch.from_numpy(case.cos_sin).cuda(), case.k_cache.clone(), case.v_cache.clone()
    ws, out = cuda_lib.Workspace(cuda_lib.OP_KV_APPEND), torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cuda_lib.dspark_kv_append(q, case.k, case.v, pos, slots, cs, K, V, q_out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(K, want[1]) and torch.equal(V, want[2])
    assert cuda_lib.dspark_read_status(ws) == (0, 0)


def test_offsets_past_32_bits(cuda_lib):
    import torch
    Hkv, page, D = 8, 64, 128
    P = (1 << 31) // (Hkv * page * D) + 5
    K = torch.zeros(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    case = Case(5, 8, Hkv, D, 128, page, 2, "bf16", seed=4)
    want = case.call(cuda_lib)
    shift = (P - 2) * page
    cuda_lib.dspark_kv_append(case.q, case.k, case.v, torch.from_numpy(case.positions).cuda(),
                              torch.from_numpy(case.slots + shift).cuda(), torch.from_numpy(case.cos_sin).cuda(), K, V)
    for s in case.slots:
        assert torch.equal(K[P - 2 + s // page, :, s % page], want[1][s // page, :, s % page])
        assert torch.equal(V[P - 2 + s // page, :, s % page], want[2][s // page, :, s % page])
    assert int((V != 0).any(dim=-1).sum()) == 5 * Hkv


def test_out_of_range_positions_and_slots_are_flagged(cuda_lib):
    import torch
    case = Case(8, 2, 2, 64, 64, 16, 3, "bf16", seed=5)
    clean = case.call(cuda_lib)
    good = case.slots.copy()
    case.slots[2], case.slots[3], case.positions[4], case.positions[5] = 48, -2, 500, -1
    ws = cuda_lib.Workspace(cuda_lib.OP_KV_APPEND)
    q, K, V = case.call(cuda_lib, workspace=ws)
    assert cuda_lib.dspark_read_status(ws)[1] & cuda_lib.STATUS_INPUT_RANGE
    keep = [0, 1, 2, 3, 6, 7]
    assert torch.equal(q[keep], clean[0][keep]) and not q[4:6].any()
    left = good.copy()
    left[[2, 3, 4, 5]] = -1
    assert torch.equal(V, _scatter(case.v_cache, case.v, left))
    for t in (0, 1, 6, 7):
        assert torch.equal(K[good[t] // 16, :, good[t] % 16], clean[1][good[t] // 16, :, good[t] % 16])
    for t in (2, 3, 4, 5):
        assert torch.equal(K[good[t] // 16, :, good[t] % 16], case.k_cache[good[t] // 16, :, good[t] % 16])


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    case = Case(4, 2, 2, 64, 64, 16, 3, "bf16", seed=6)
    pos, slots, cs = (torch.from_numpy(x).cuda() for x in (case.positions, case.slots, case.cos_sin))

    def call(q=case.q, k=case.k, v=case.v, pos=pos, slots=slots, cs=cs, K=case.k_cache, V=case.v_cache, **kw):
        return ds.dspark_kv_append(q, k, v, pos, slots, cs, K, V, **kw)

    with pytest.raises(TypeError):
        call(k=case.k.float())
    with pytest.raises(TypeError):
        call(q=case.q.half())
    with pytest.raises(TypeError):
        call(slots=slots.long())
    with pytest.raises(ValueError):
        call(slots=slots[:3])
    with pytest.raises(ValueError):
        call(k=case.k.transpose(0, 1), v=case.v.transpose(0, 1))
    with pytest.raises(ValueError):
        call(K=case.k_cache[:2])
    with pytest.raises(ValueError):
        call(k_norm=torch.ones(32, device="cuda"))
    for kw in (dict(cs=cs[:, :40].contiguous()), dict(cs=torch.ones(5, 128, device="cuda")), dict(q_out=case.q)):
        with pytest.raises((ds.DSparkError, ValueError)):
            call(**kw)
