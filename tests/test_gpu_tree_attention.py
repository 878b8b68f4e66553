"""GPU parity: attention of a tree of drafted tokens over a paged cache, against the 64-bit oracle.

Every cache slot that holds no token is NaN, so a read past a request's length shows.
"""
import math

import numpy as np
import pytest

from tests._serving import ULP, PagedCase
from tests._trees import TreeCase, random_parents

pytestmark = pytest.mark.gpu


def _tree(B, N, *args, shape="random", seed=0, **kw):
    parents = random_parents(np.random.default_rng(seed + 1), B, N, deepest=9 if shape == "random" else None, shape=shape)
    return TreeCase(B, N, *args, parents=parents, seed=seed, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G,Hkv", [(1, 1, 2), (3, 3, 2), (8, 4, 2), (17, 4, 1), (33, 1, 2), (31, 2, 1), (64, 4, 1), (70, 3, 1)])
def test_heads_nodes_and_types(cuda_lib, dtype, D, N, G, Hkv):
    lens = [N, N + 1, max(N, 127), max(N, 128), max(N, 129), 300]
    case = _tree(len(lens), N, G * Hkv, Hkv, D, 16, lens, dtype=dtype, seed=N * 100 + G)
    case.check(cuda_lib, rows=250)
    case.window, case.sinks = N + 20, 3
    case.check(cuda_lib, rows=250)


@pytest.mark.parametrize("shape", ["chain", "star", "forest", "random"])
@pytest.mark.parametrize("N", [2, 32, 33, 65, 128, 130, 255, 256])
def test_shapes_of_trees_and_word_ends(cuda_lib, N, shape):
    """The tree begins at every place of a 32-token word and may reach over three tiles."""
    lens = [N, N + 31, N + 32, N + 100, N + 127, N + 128, N + 200, 700]
    case = _tree(len(lens), N, 2, 1, 64, 32, lens, shape=shape, seed=N)
    case.check(cuda_lib, rows=400)
    case.window, case.sinks = N, 40
    case.check(cuda_lib, rows=200)


def test_a_chain_equals_a_causal_window(cuda_lib):
    import torch
    lens = [40, 17, 300, 1000, 129]
    case = _tree(5, 17, 8, 2, 128, 16, lens, shape="chain", seed=3)
    plain = PagedCase(5, 17, 8, 2, 128, 16, lens, seed=3)
    a, la = case.run(cuda_lib, lengths=[17, 3, 0, 17, 9])
    b, lb = plain.run(cuda_lib, lengths=[17, 3, 0, 17, 9])
    assert torch.equal(a, b) and torch.equal(la, lb)          # the same sums in the same order
    case.window, case.sinks = 2000, 5                         # a window wider than any request
    a, la = case.run(cuda_lib, lengths=[17, 3, 0, 17, 9])
    assert float((a.float() - b.float()).abs().max()) <= 2 * ULP["bf16"] * 6 and float((la[3] - lb[3]).abs().max()) < 1e-5


@pytest.mark.parametrize("page", [8, 16, 64, 256])
def test_pages_and_windows_around_their_ends(cuda_lib, page):
    lens = [12, page + 12, 2 * page + 3 + 12, 127 + 12, 128 + 12, 140 + 12, 513, 1200]
    case = _tree(len(lens), 12, 8, 2, 128, page, lens, seed=page)
    case.check(cuda_lib, rows=100)
    for window, sinks in ((12, 0), (13, 1), (128, 128), (129, 127), (100, 300), (500, 129), (4000, 7)):
        case.window, case.sinks = window, sinks
        case.check(cuda_lib, rows=100)


def test_ragged_trees_and_empty_requests(cuda_lib):
    lens = [0, 6, 30, 40, 1, 200, 64]
    lengths = [0, 6, 6, 0, 1, 4, 2]
    case = _tree(len(lens), 6, 8, 2, 64, 16, lens, seed=5)
    for window in (0, 9):
        case.window = window
        out, lse = case.check(cuda_lib, lengths=lengths)
        assert not out[0].any() and bool((lse[0] == -math.inf).all())
        assert not out[3].any() and not out[4, 1:].any() and not out[5, 4:].any()


@pytest.mark.parametrize("B,N,L,window", [(1, 25, 5000, 0), (1, 25, 40001, 0), (1, 64, 9000, 4000), (3, 40, 20000, 0), (2, 200, 7001, 900)])
def test_long_contexts_are_split_and_joined(cuda_lib, B, N, L, window):
    lens = [max(N, L - 777 * b) for b in range(B)]
    case = _tree(B, N, 8, 2, 128, 64, lens, seed=L, gain=2.0, window=window, sinks=4)
    case.check(cuda_lib, rows=16)


@pytest.mark.parametrize("B", [37, 300, 1100])
def test_many_requests_of_mixed_lengths(cuda_lib, B):
    rng = np.random.default_rng(B)
    lens = 5 + np.exp(rng.uniform(0, math.log(900), B)).astype(int)
    lengths = rng.integers(0, 6, B)
    case = _tree(B, 5, 16, 4, 64, 32, lens.tolist(), dtype="f16", seed=B)
    for window in (0, 64):
        case.window, case.sinks = window, 2
        case.check(cuda_lib, lengths=lengths.tolist(), rows=150)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("N,G", [(5, 2), (12, 4), (20, 5), (40, 4), (61, 5)])
def test_infinities_and_nan_reach_only_rows_that_see_them(cuda_lib, dtype, bad, N, G):
    import torch
    lens = [200, 131, 64]
    case = _tree(3, N, 2 * G, 2, 128, 16, lens, dtype=dtype, seed=11)
    case.parents[0, :5] = [-1, 0, 0, 1, 2]                    # node 1 is seen by itself, 3 and what hangs from them
    clean, clean_lse = case.run(cuda_lib)
    j = lens[0] - N + 1
    at = (int(case.table[0, j // 16]), 0, j % 16)
    keep = case.v[at].clone()
    case.v[at][5] = bad
    out, lse = case.run(cuda_lib)
    hit = torch.tensor([j in case.sees(0, i, None, True) for i in range(N)], device="cuda")
    assert bool(hit[1]) and bool(hit[3]) and not bool(hit[[0, 2, 4]].any())
    assert torch.equal(out[0, ~hit], clean[0, ~hit]) and torch.equal(lse, clean_lse)
    assert torch.equal(out[1:], clean[1:]) and torch.equal(out[0, :, G:], clean[0, :, G:])
    got = out[0, hit][:, :G, 5].float()
    assert bool(got.isnan().all()) if math.isnan(bad) else bool((got == bad).all())
    rest = [d for d in range(128) if d != 5]
    assert float((out[0][..., rest].float() - clean[0][..., rest].float()).abs().max()) <= 4 * ULP[dtype] * 3
    case.v[at] = keep
    case.k[at] = bad
    out2, lse2 = case.run(cuda_lib)
    assert torch.equal(out2[0, ~hit], clean[0, ~hit]) and torch.equal(lse2[0, ~hit], clean_lse[0, ~hit])
    assert torch.equal(out2[1:], clean[1:])


def test_pages_behind_the_window_are_not_read(cuda_lib):
    """Their entries of the table may be anything, their pages may hold anything."""
    import torch
    lens = [1000, 777]
    case = _tree(2, 12, 8, 2, 128, 16, lens, seed=31, window=100, sinks=20)
    ws = cuda_lib.Workspace(cuda_lib.OP_TREE_ATTENTION, 2, 12, 8, 128)
    out, lse = case.check(cuda_lib, workspace=ws)
    for b, L in enumerate(lens):
        last = (L - 12 - 100 + 1) // 16                       # the first page that a row may see, behind the sinks'
        for p in range(2, last):
            case.k[int(case.table[b, p])] = math.nan
            case.v[int(case.table[b, p])] = math.nan
            case.table[b, p] = (-1, 10 ** 6)[p % 2]
    again, lse2 = case.run(cuda_lib, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert cuda_lib.dspark_read_status(ws) == (0, 0)


def test_repeats_bit_for_bit_and_on_another_stream(cuda_lib):
    import torch
    case = _tree(3, 25, 16, 4, 128, 16, [3000, 1200, 77], seed=17)
    ws = cuda_lib.Workspace(cuda_lib.OP_TREE_ATTENTION, 3, 25, 16, 128)
    ws.buf.fill_(255)
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
    case = _tree(2, 9, 8, 2, 64, 16, [500, 33], seed=19)
    ws = cuda_lib.Workspace(cuda_lib.OP_TREE_ATTENTION, 2, 9, 8, 64)
    table, kv = torch.from_numpy(case.table).cuda(), torch.from_numpy(case.kv_len).cuda()
    parents = torch.from_numpy(case.parents).cuda()
    out, lse = torch.empty_like(case.q), torch.empty(2, 9, 8, device="cuda")

    def call():
        cuda_lib.dspark_tree_attention(case.q, case.k, case.v, table, kv, parents, case.scale, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    kv.copy_(torch.tensor([123, 20], dtype=torch.int32))      # lengths and trees are read when the graph runs
    case.kv_len = np.array([123, 20], np.int32)
    case.parents = random_parents(np.random.default_rng(99), 2, 9)
    parents.copy_(torch.from_numpy(case.parents))
    g.replay()
    torch.cuda.synchronize()
    eager, elsew = case.run(cuda_lib)
    assert torch.equal(out, eager) and torch.equal(lse, elsew)


def test_out_of_range_values_are_flagged(cuda_lib):
    import torch
    ds = cuda_lib
    case = _tree(4, 5, 4, 2, 64, 16, [60, 50, 40, 30], seed=23)
    clean, _ = case.run(ds)
    ws = ds.Workspace(ds.OP_TREE_ATTENTION, 4, 5, 4, 64)
    case.kv_len = np.array([60, 10 ** 6, -1, 30], np.int32)
    out, lse = case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert not out[1:3].any() and bool((lse[1:3] == -math.inf).all())
    case.kv_len = np.array([60, 4, 40, 30], np.int32)         # fewer tokens than nodes
    out, _ = case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
    assert not out[1].any() and torch.equal(out[2:], clean[2:])
    case.kv_len = np.array([60, 50, 40, 30], np.int32)
    out, _ = case.run(ds, lengths=[5, 6, -1, 5], workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and not out[1:3].any()
    good = case.parents.copy()
    for value in (2, 3, 10 ** 6, -2, -2 ** 31):               # not before node 2, or below -1: read as -1
        case.parents = good.copy()
        case.parents[1, 2] = value
        out, _ = case.run(ds, workspace=ws)
        assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
        case.parents[1, 2] = -1
        case.check(ds)
        assert torch.equal(out, case.run(ds, workspace=ws)[0])
        assert ds.dspark_read_status(ws) == (0, 0)
    case.parents = good
    first = int(case.table[1, 0])
    case.table[1, 0] = 10 ** 6
    out, _ = case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2:], clean[2:])
    case.table[1, 0] = first
    case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws) == (0, 0)


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    case = _tree(2, 4, 4, 2, 64, 16, [20, 30], seed=29)
    dev = lambda x: torch.from_numpy(x).cuda()
    table, kv, parents = dev(case.table), dev(case.kv_len), dev(case.parents)

    def call(q=case.q, k=case.k, v=case.v, table=table, kv=kv, parents=parents, scale=0.1, **kw):
        return ds.dspark_tree_attention(q, k, v, table, kv, parents, scale, **kw)

    call()
    for bad in (dict(q=case.q.float()), dict(k=case.k.half()), dict(kv=kv.long()), dict(parents=parents.long()), dict(parents=None)):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(parents=parents[:, :3].contiguous()), dict(parents=parents[:1]), dict(parents=parents.T), dict(table=table[:1]),
                dict(lse=torch.empty(2, 4, 5, device="cuda")), dict(lengths=kv[:1])):
        with pytest.raises(ValueError):
            call(**bad)
    small = ds.Workspace(ds.OP_PAGED_ATTENTION, 2, 4, 4, 64)
    for bad in (dict(scale=math.nan), dict(window=3), dict(window=-1), dict(sinks=-1), dict(workspace=small)):
        with pytest.raises(ds.DSparkError) as e:
            call(**bad)
        assert e.value.status == 1
    with pytest.raises(ds.DSparkError):
        ds.dspark_tree_attention(torch.zeros(1, 257, 2, 64, dtype=torch.bfloat16, device="cuda"), case.k, case.v, table[:1], kv[:1],
                                 torch.zeros(1, 257, dtype=torch.int32, device="cuda"), 0.1)


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^31 values: the last pages hold the request."""
    import torch
    Hkv, page, D = 8, 64, 128
    P = (1 << 31) // (Hkv * page * D) + 40
    k = torch.zeros(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = _tree(1, 20, 16, Hkv, D, page, [500], seed=31, window=300, sinks=4)
    table = torch.arange(P - 8, P, dtype=torch.int32, device="cuda")[None].contiguous()
    for dst, src in ((k, small.k), (v, small.v)):
        dst[P - 8:] = src[small.table[0, :8]]
    kv, parents = torch.from_numpy(small.kv_len).cuda(), torch.from_numpy(small.parents).cuda()
    out = cuda_lib.dspark_tree_attention(small.q, k, v, table, kv, parents, small.scale, window=300, sinks=4)
    assert torch.equal(out, small.run(cuda_lib)[0])
