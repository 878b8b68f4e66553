"""GPU parity: attention of a window of new tokens over a paged cache, against the 64-bit oracle.

Every cache slot that holds no token is NaN, so a read past a request's length shows.
"""
import math

import numpy as np
import pytest

from tests._serving import ULP, PagedCase, half_dtype

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G,Hkv", [(1, 1, 2), (1, 4, 2), (1, 8, 1), (3, 3, 2), (8, 4, 2), (9, 7, 1), (17, 4, 1),
                                     (33, 1, 2), (33, 4, 1), (2, 65, 1), (1, 128, 1)])
def test_heads_windows_and_types(cuda_lib, dtype, D, N, G, Hkv):
    lens = [N, 1, 127, 128, 129, 300]
    case = PagedCase(len(lens), N, G * Hkv, Hkv, D, 16, lens, dtype, seed=N * 100 + G)
    for causal in (True, False):
        case.check(cuda_lib, causal=causal, rows=250)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_page_sizes_and_lengths_around_their_ends(cuda_lib, page):
    lens = [1, page - 1, page, page + 1, 2 * page + 3, 128 - 1, 128, 129, 255, 257, 513]
    case = PagedCase(len(lens), 2, 8, 2, 128, page, lens, seed=page)
    case.check(cuda_lib, rows=120)
    case.check(cuda_lib, causal=False, rows=60)


def test_ragged_windows_empty_requests_and_windows_longer_than_the_cache(cuda_lib):
    lens = [0, 5, 3, 40, 1, 200, 64]
    lengths = [0, 6, 6, 0, 1, 4, 2]              # 6 new tokens over 5 or 3 cached: the first rows see nothing
    case = PagedCase(len(lens), 6, 8, 2, 64, 16, lens, seed=5)
    for causal in (True, False):
        out, lse = case.check(cuda_lib, lengths=lengths, causal=causal)
        assert not out[0].any() and bool((lse[0] == -math.inf).all())
        assert not out[3].any() and not out[4, 1:].any()


@pytest.mark.parametrize("B,N,L", [(1, 1, 1), (1, 1, 5000), (1, 1, 40001), (1, 5, 9000), (3, 1, 20000), (2, 17, 7001)])
def test_long_contexts_are_split_and_joined(cuda_lib, B, N, L):
    lens = [max(1, L - 777 * b) for b in range(B)]
    case = PagedCase(B, N, 8, 2, 128, 64, lens, seed=L, gain=2.0)
    case.check(cuda_lib, rows=12)


@pytest.mark.parametrize("B", [1, 37, 300])
def test_many_requests_of_mixed_lengths(cuda_lib, B):
    rng = np.random.default_rng(B)
    lens = np.exp(rng.uniform(0, math.log(900), B)).astype(int).clip(1)
    case = PagedCase(B, 4, 16, 4, 64, 32, lens, "f16", seed=B)
    case.check(cuda_lib, lengths=[min(4, L) for L in lens], rows=80)


def test_scores_that_grow_and_that_are_large(cuda_lib):
    """Keys ordered so that the running maximum rises many times, by little and by a lot."""
    import torch
    case = PagedCase(2, 2, 4, 1, 128, 16, [900, 700], seed=9)
    for b in range(2):
        j = np.arange(case.kv_len[b])
        pages, offs = case.table[b, j // 16], j % 16
        ramp = torch.linspace(0.01, 4.0, len(j), device="cuda")[:, None] * case.q[b, 0, 0].float()
        case.k[pages, 0, offs] = ramp.to(case.k.dtype)
    case.check(cuda_lib)
    case.scale = -case.scale                       # the largest first, the tail vanishing
    case.check(cuda_lib)
    case.scale = 0.0
    case.check(cuda_lib)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("N,G", [(3, 2), (12, 4), (20, 5)])
def test_infinities_and_nan_reach_only_rows_that_see_them(cuda_lib, dtype, bad, N, G):
    import torch
    lens = [200, 131, 64]
    case = PagedCase(3, N, 2 * G, 2, 128, 16, lens, dtype, seed=11)
    clean, clean_lse = case.run(cuda_lib)
    # the second new token of request 0: rows 1.. see it, row 0 does not
    j = lens[0] - N + 1
    at = (int(case.table[0, j // 16]), 0, j % 16)
    keep = case.v[at].clone()
    case.v[at][5] = bad
    out, lse = case.run(cuda_lib)
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(lse, clean_lse)
    assert torch.equal(out[1:], clean[1:]) and torch.equal(out[0, :, G:], clean[0, :, G:])
    hit = out[0, 1:, :G, 5].float()
    assert bool(hit.isnan().all()) if math.isnan(bad) else bool((hit == bad).all())
    rest = [d for d in range(128) if d != 5]
    case.v[at] = keep
    # other values of the rows that see it: as without it
    tol = 4 * ULP[dtype] * 3
    assert float((out[0][..., rest].float() - clean[0][..., rest].float()).abs().max()) <= tol
    # an infinite or NaN key reaches the rows that see it and no others
    case.k[at] = bad
    out2, lse2 = case.run(cuda_lib)
    assert torch.equal(out2[0, 0], clean[0, 0]) and torch.equal(lse2[0, 0], clean_lse[0, 0])
    assert torch.equal(out2[1:], clean[1:])


def test_a_key_that_scores_minus_infinity_has_no_weight(cuda_lib):
    """-infinity in one value of a key against a positive query value: the score is -infinity."""
    import torch
    case = PagedCase(1, 1, 1, 1, 64, 16, [40], seed=13)
    case.q[0, 0, 0, 3] = 1.0
    for j in range(0, 40, 2):
        case.k[int(case.table[0, j // 16]), 0, j % 16, 3] = -math.inf
    case.check(cuda_lib)
    for j in range(40):
        case.k[int(case.table[0, j // 16]), 0, j % 16, 3] = -math.inf
    out, lse = case.run(cuda_lib)
    assert not out.any() and float(lse[0, 0, 0]) == -math.inf


def test_repeats_bit_for_bit_and_on_another_stream(cuda_lib):
    import torch
    case = PagedCase(3, 5, 16, 4, 128, 16, [3000, 1200, 77], seed=17)
    ws = cuda_lib.Workspace(cuda_lib.OP_PAGED_ATTENTION, 3, 5, 16, 128)
    ws.buf.fill_(255)                              # a workspace holds anything before a call
    a, la = case.run(cuda_lib, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(5):
            b, lb = case.run(cuda_lib, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert cuda_lib.dspark_read_status(ws) == (0, 0)


def test_capture_and_replay(cuda_lib):
    import torch
    case = PagedCase(2, 3, 8, 2, 64, 16, [500, 33], seed=19)
    ws = cuda_lib.Workspace(cuda_lib.OP_PAGED_ATTENTION, 2, 3, 8, 64)
    table, kv = torch.from_numpy(case.table).cuda(), torch.from_numpy(case.kv_len).cuda()
    out, lse = torch.empty_like(case.q), torch.empty(2, 3, 8, device="cuda")

    def call():
        cuda_lib.dspark_paged_attention(case.q, case.k, case.v, table, kv, case.scale, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    kv.copy_(torch.tensor([123, 20], dtype=torch.int32))       # the lengths are read when the graph runs
    case.kv_len = np.array([123, 20], np.int32)
    g.replay()
    torch.cuda.synchronize()
    eager, elsew = case.run(cuda_lib)
    assert torch.equal(out, eager) and torch.equal(lse, elsew)


def test_out_of_range_lengths_and_pages_are_flagged(cuda_lib):
    import torch
    case = PagedCase(4, 2, 4, 2, 64, 16, [60, 50, 40, 30], seed=23)
    clean, _ = case.run(cuda_lib)
    ws = cuda_lib.Workspace(cuda_lib.OP_PAGED_ATTENTION, 4, 2, 4, 64)
    case.kv_len = np.array([60, 10 ** 6, -1, 30], np.int32)
    out, lse = case.run(cuda_lib, workspace=ws)
    assert cuda_lib.dspark_read_status(ws)[1] & cuda_lib.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert not out[1:3].any() and bool((lse[1:3] == -math.inf).all())
    case.kv_len = np.array([60, 50, 40, 30], np.int32)
    out, lse = case.run(cuda_lib, lengths=[2, 3, -1, 2], workspace=ws)
    assert cuda_lib.dspark_read_status(ws)[1] & cuda_lib.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and not out[1:3].any()
    first = int(case.table[1, 0])
    case.table[1, 0] = 10 ** 6
    out, _ = case.run(cuda_lib, workspace=ws)
    assert cuda_lib.dspark_read_status(ws)[1] & cuda_lib.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2:], clean[2:])
    case.table[1, 0] = first
    case.run(cuda_lib, workspace=ws)
    assert cuda_lib.dspark_read_status(ws) == (0, 0)


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    case = PagedCase(2, 2, 4, 2, 64, 16, [20, 30], seed=29)
    table, kv = torch.from_numpy(case.table).cuda(), torch.from_numpy(case.kv_len).cuda()

    def call(q=case.q, k=case.k, v=case.v, table=table, kv=kv, scale=0.1, **kw):
        return ds.dspark_paged_attention(q, k, v, table, kv, scale, **kw)

    with pytest.raises(TypeError):
        call(q=case.q.float())
    with pytest.raises(TypeError):
        call(k=case.k.to(half_dtype("f16")))
    with pytest.raises(TypeError):
        call(kv=kv.long())
    with pytest.raises(ValueError):
        call(q=case.q.transpose(0, 1))
    with pytest.raises(ValueError):
        call(table=table[:1].contiguous())
    with pytest.raises(ValueError):
        call(lse=torch.empty(2, 2, 5, device="cuda"))
    small = ds.Workspace(ds.OP_PAGED_ATTENTION, 2, 2, 4, 64)
    small.nbytes = 128
    for bad in (dict(scale=math.inf), dict(q=case.q[:, :, :3].contiguous()),
                dict(k=torch.zeros(3, 2, 24, 64, dtype=torch.bfloat16, device="cuda"),
                     v=torch.zeros(3, 2, 24, 64, dtype=torch.bfloat16, device="cuda")),
                dict(q=case.q[..., :32].contiguous(), k=case.k[..., :32].contiguous(), v=case.v[..., :32].contiguous()),
                dict(workspace=small)):
        with pytest.raises(ds.DSparkError) as e:
            call(**bad)
        assert e.value.status == 1


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^31 values: the last pages hold the request."""
    import torch
    Hkv, page, D = 8, 64, 128
    P = (1 << 31) // (Hkv * page * D) + 40
    k = torch.zeros(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = PagedCase(1, 2, 16, Hkv, D, page, [500], seed=31)
    table = torch.arange(P - 8, P, dtype=torch.int32, device="cuda")[None].contiguous()
    for dst, src in ((k, small.k), (v, small.v)):
        dst[P - 8:] = src[small.table[0, :8]]
    kv = torch.from_numpy(small.kv_len).cuda()
    out = cuda_lib.dspark_paged_attention(small.q, k, v, table, kv, small.scale)
    assert torch.equal(out, small.run(cuda_lib)[0])
