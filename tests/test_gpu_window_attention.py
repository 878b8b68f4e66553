"""GPU parity: attention with a sliding window and sinks over a paged cache, against the 64-bit oracle."""
import math

import numpy as np
import pytest

from tests._serving import PagedCase
from tests._trees import WindowCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G,Hkv", [(1, 1, 2), (1, 4, 2), (1, 8, 1), (3, 3, 2), (17, 4, 1), (33, 1, 2), (40, 4, 1), (2, 65, 1), (1, 128, 1)])
def test_heads_windows_and_types(cuda_lib, dtype, D, N, G, Hkv):
    lens = [N, 1, 127, 128, 129, 300, 520]
    case = WindowCase(len(lens), N, G * Hkv, Hkv, D, 16, lens, dtype, seed=N * 100 + G, window=50, sinks=3)
    for causal in (True, False):
        case.check(cuda_lib, causal=causal, rows=250)


@pytest.mark.parametrize("window", [1, 2, 31, 127, 128, 129, 200, 256, 500, 10 ** 9])
@pytest.mark.parametrize("sinks", [0, 1, 127, 128, 129, 400, 2 ** 31 - 1])
def test_windows_and_sinks_around_tile_ends(cuda_lib, window, sinks):
    lens = [1, 128, 129, 130, 255, 256, 257, 384, 385, 500, 900]
    case = WindowCase(len(lens), 5, 4, 2, 64, 16, lens, seed=window % 1000 + sinks % 1000, window=window, sinks=sinks)
    case.check(cuda_lib, rows=120)
    case.check(cuda_lib, causal=False, rows=120)


@pytest.mark.parametrize("page", [8, 32, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_of_a_prompt(cuda_lib, page, causal):
    """More new tokens than a row tile holds, with the first tokens of the request among them."""
    lens = [300, 700, 301]
    case = WindowCase(3, 300, 4, 2, 64, page, lens, "f16", seed=page, window=90, sinks=5)
    case.check(cuda_lib, lengths=[300, 200, 1], causal=causal, rows=300)
    case.window, case.sinks = 257, 0
    case.check(cuda_lib, causal=causal, rows=300)


def test_a_wide_window_equals_none(cuda_lib):
    import torch
    lens = [40, 17, 300, 1000, 129]
    case = WindowCase(5, 17, 8, 2, 128, 16, lens, seed=3, window=1000, sinks=0)
    plain = PagedCase(5, 17, 8, 2, 128, 16, lens, seed=3)
    for causal in (True, False):
        a, la = case.run(cuda_lib, lengths=[17, 3, 0, 17, 9], causal=causal)
        b, lb = plain.run(cuda_lib, lengths=[17, 3, 0, 17, 9], causal=causal)
        case.check(cuda_lib, lengths=[17, 3, 0, 17, 9], causal=causal, rows=100)
        torch.testing.assert_close(la, lb, rtol=0, atol=1e-5)


def test_ragged_windows_empty_requests_and_windows_longer_than_the_cache(cuda_lib):
    lens = [0, 5, 3, 40, 1, 200, 64]
    lengths = [0, 6, 6, 0, 1, 4, 2]
    case = WindowCase(len(lens), 6, 8, 2, 64, 16, lens, seed=5, window=4, sinks=1)
    for causal in (True, False):
        out, lse = case.check(cuda_lib, lengths=lengths, causal=causal)
        assert not out[0].any() and bool((lse[0] == -math.inf).all())
        assert not out[3].any() and not out[4, 1:].any()


@pytest.mark.parametrize("B,N,L,window", [(1, 1, 5000, 4000), (1, 1, 40001, 30000), (1, 5, 9000, 8999), (3, 1, 20000, 7777), (1, 900, 4001, 1500)])
def test_long_windows_are_split_and_joined(cuda_lib, B, N, L, window):
    lens = [max(1, L - 777 * b) for b in range(B)]
    case = WindowCase(B, N, 8, 2, 128, 64, lens, seed=L, gain=2.0, window=window, sinks=130)
    case.check(cuda_lib, rows=16)


@pytest.mark.parametrize("B", [64, 300, 1100])
def test_many_requests_of_mixed_lengths(cuda_lib, B):
    rng = np.random.default_rng(B)
    lens = np.exp(rng.uniform(0, math.log(1500), B)).astype(int).clip(1)
    lens[rng.random(B) < 0.05] = 0
    case = WindowCase(B, 3, 16, 4, 64, 32, lens.tolist(), "f16", seed=B, window=130, sinks=4)
    lengths = np.minimum(rng.integers(0, 4, B), lens)
    case.check(cuda_lib, lengths=lengths.tolist(), rows=150)
    case.check(cuda_lib, lengths=lengths.tolist(), causal=False, rows=150)


def test_scores_that_grow_scales_below_zero_and_of_zero(cuda_lib):
    import torch
    case = WindowCase(2, 2, 4, 1, 128, 16, [900, 700], seed=9, window=400, sinks=9)
    for b in range(2):
        j = np.arange(case.kv_len[b])
        pages, offs = case.table[b, j // 16], j % 16
        ramp = torch.linspace(0.01, 4.0, len(j), device="cuda")[:, None] * case.q[b, 0, 0].float()
        case.k[pages, 0, offs] = ramp.to(case.k.dtype)
    case.check(cuda_lib)
    case.scale = -case.scale
    case.check(cuda_lib)
    case.scale = 0.0
    case.check(cuda_lib)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("N,G", [(3, 2), (12, 4), (20, 5), (40, 4), (61, 5)])
def test_infinities_and_nan_reach_only_rows_that_see_them(cuda_lib, dtype, bad, N, G):
    """A value in the tile where the window begins: the first rows see it, the later ones do not."""
    import torch
    lens = [400, 131, 64]
    case = WindowCase(3, N, 2 * G, 2, 128, 16, lens, dtype, seed=11, window=60, sinks=2)
    clean, clean_lse = case.run(cuda_lib)
    j = lens[0] - N - 60 + 2                                  # rows 0 and 1 see it
    at = (int(case.table[0, j // 16]), 0, j % 16)
    keep = case.v[at].clone()
    case.v[at][5] = bad
    out, lse = case.run(cuda_lib)
    hit = torch.tensor([j in case.sees(0, i, None, True) for i in range(N)], device="cuda")
    assert hit.tolist() == [True, True] + [False] * (N - 2)
    assert torch.equal(out[0, ~hit], clean[0, ~hit]) and torch.equal(lse, clean_lse)
    assert torch.equal(out[1:], clean[1:]) and torch.equal(out[0, :, G:], clean[0, :, G:])
    got = out[0, hit][:, :G, 5].float()
    assert bool(got.isnan().all()) if math.isnan(bad) else bool((got == bad).all())
    case.v[at] = keep
    case.k[at] = bad
    out2, lse2 = case.run(cuda_lib)
    assert torch.equal(out2[0, ~hit], clean[0, ~hit]) and torch.equal(lse2[0, ~hit], clean_lse[0, ~hit])
    assert torch.equal(out2[1:], clean[1:])


def test_pages_out_of_the_window_are_not_read(cuda_lib):
    import torch
    lens = [1000, 777, 300]
    for N in (1, 40):
        case = WindowCase(3, N, 8, 2, 128, 16, lens, seed=31, window=100, sinks=20)
        ws = cuda_lib.Workspace(cuda_lib.OP_WINDOW_ATTENTION, 3, N, 8, 128)
        out, lse = case.check(cuda_lib, workspace=ws, rows=100)
        for b, L in enumerate(lens):
            for p in range(2, (L - N - 100 + 1) // 16):
                case.k[int(case.table[b, p])] = math.nan
                case.v[int(case.table[b, p])] = math.inf
                case.table[b, p] = (-1, 10 ** 6)[p % 2]
        again, lse2 = case.run(cuda_lib, workspace=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
        assert cuda_lib.dspark_read_status(ws) == (0, 0)


def test_stream_capture_and_workspaces(cuda_lib):
    import torch
    case = WindowCase(2, 3, 8, 2, 64, 16, [500, 33], seed=19, window=40, sinks=2)
    ws = cuda_lib.Workspace(cuda_lib.OP_WINDOW_ATTENTION, 2, 3, 8, 64)
    ws.buf.fill_(255)
    table, kv = torch.from_numpy(case.table).cuda(), torch.from_numpy(case.kv_len).cuda()
    out, lse = torch.empty_like(case.q), torch.empty(2, 3, 8, device="cuda")

    def call():
        cuda_lib.dspark_window_attention(case.q, case.k, case.v, table, kv, 40, 2, case.scale, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    kv.copy_(torch.tensor([123, 20], dtype=torch.int32))
    case.kv_len = np.array([123, 20], np.int32)
    g.replay()
    torch.cuda.synchronize()
    eager, elsew = case.run(cuda_lib)
    assert torch.equal(out, eager) and torch.equal(lse, elsew)
    assert cuda_lib.dspark_read_status(ws) == (0, 0)


def test_out_of_range_values_are_flagged(cuda_lib):
    import torch
    ds = cuda_lib
    case = WindowCase(4, 2, 4, 2, 64, 16, [60, 50, 40, 30], seed=23, window=30, sinks=1)
    clean, _ = case.run(ds)
    ws = ds.Workspace(ds.OP_WINDOW_ATTENTION, 4, 2, 4, 64)
    case.kv_len = np.array([60, 10 ** 6, -1, 30], np.int32)
    out, lse = case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert not out[1:3].any() and bool((lse[1:3] == -math.inf).all())
    case.kv_len = np.array([60, 50, 40, 30], np.int32)
    out, _ = case.run(ds, lengths=[2, 3, -1, 2], workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and not out[1:3].any()
    last = int(case.table[1, 2])
    case.table[1, 2] = 10 ** 6
    out, _ = case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2:], clean[2:])
    case.table[1, 2] = last
    case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws) == (0, 0)


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    case = WindowCase(2, 2, 4, 2, 64, 16, [20, 30], seed=29, window=8, sinks=2)
    table, kv = torch.from_numpy(case.table).cuda(), torch.from_numpy(case.kv_len).cuda()

    def call(q=case.q, k=case.k, table=table, kv=kv, window=8, sinks=2, scale=0.1, **kw):
        return ds.dspark_window_attention(q, k, case.v, table, kv, window, sinks, scale, **kw)

    call()
    for bad in (dict(q=case.q.float()), dict(k=case.k.half()), dict(kv=kv.long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=case.q.transpose(0, 1)), dict(table=table[:1]), dict(lse=torch.empty(2, 2, 5, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=math.inf)):
        with pytest.raises(ds.DSparkError) as e:
            call(**bad)
        assert e.value.status == 1
