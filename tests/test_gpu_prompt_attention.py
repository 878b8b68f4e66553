"""GPU parity: attention within packed prompts against the 64-bit oracle."""
import math

import numpy as np
import pytest

import oracle
from tests._serving import ULP, check_attention, f64, half_dtype

pytestmark = pytest.mark.gpu


def _inputs(T, Hq, Hkv, D, dtype, seed, gain=1.0, fused=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda")
    rows[:, :Hq * D] *= gain
    rows = rows.to(half_dtype(dtype))
    q, k, v = rows.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    q, k, v = q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D)
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _run(ds, q, k, v, cu, causal=True, scale=None, **kw):
    import torch
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = ds.dspark_prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                     q.shape[2] ** -0.5 if scale is None else scale, causal=causal, lse=lse, **kw)
    return out, lse


def _check(ds, q, k, v, cu, dtype, causal=True, rows=200, seed=0, scale=None):
    import torch
    out, lse = _run(ds, q, k, v, cu, causal, scale)
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    pick = np.random.default_rng(seed).choice(T * Hq, min(rows, T * Hq), replace=False)
    seq = np.searchsorted(cu, np.arange(T), side="right") - 1
    ref = []
    for r in pick:
        t, h = int(r) // Hq, int(r) % Hq
        if seq[t] < 0 or seq[t] >= len(cu) - 1:
            a = z = 0
        else:
            a, z = cu[seq[t]], (t + 1 if causal else cu[seq[t] + 1])
        ref.append(oracle.attend_row(f64(q[t, h]), f64(k[a:z, h // group]).reshape(z - a, D),
                                     f64(v[a:z, h // group]).reshape(z - a, D),
                                     D ** -0.5 if scale is None else scale))
    at = torch.from_numpy(pick).cuda()
    check_attention(out.view(T * Hq, D)[at], lse.view(-1)[at], [np.array(x) for x in zip(*ref)], dtype, T, 6.0)
    return out, lse


def _cu(lens):
    return [0] + np.cumsum(lens).tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 2), (6, 2), (5, 1), (16, 2), (7, 1), (64, 1), (128, 1)])
def test_heads_and_types(cuda_lib, dtype, D, Hq, Hkv):
    lens = [1, 130, 7, 257, 64]
    q, k, v = _inputs(sum(lens), Hq, Hkv, D, dtype, Hq * 10 + Hkv)
    for causal in (True, False):
        _check(cuda_lib, q, k, v, _cu(lens), dtype, causal)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 700])
def test_lengths_around_tiles(cuda_lib, n):
    q, k, v = _inputs(n, 8, 2, 128, "bf16", n, fused=n % 2 == 0)
    for causal in (True, False):
        _check(cuda_lib, q, k, v, [0, n], "bf16", causal, rows=100)


def test_empty_sequences_and_tokens_outside(cuda_lib):
    import torch
    cu = [3, 3, 40, 40, 41, 300, 300]
    q, k, v = _inputs(310, 4, 2, 64, "bf16", 3)
    for causal in (True, False):
        out, lse = _check(cuda_lib, q, k, v, cu, "bf16", causal, rows=400)
        assert not out[:3].any() and not out[300:].any()
        assert bool((lse[:3] == -math.inf).all()) and bool((lse[300:] == -math.inf).all())
    out, lse = _run(cuda_lib, q, k, v, [0, 0])
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("causal", [True, False])
def test_long_and_many(cuda_lib, causal):
    q, k, v = _inputs(5003, 8, 2, 128, "bf16", 5, gain=2.0)
    _check(cuda_lib, q, k, v, [0, 5003], "bf16", causal, rows=40)
    rng = np.random.default_rng(6)
    lens = np.exp(rng.uniform(0, math.log(400), 60)).astype(int).clip(1).tolist()
    q, k, v = _inputs(sum(lens), 12, 4, 64, "f16", 7)
    _check(cuda_lib, q, k, v, _cu(lens), "f16", causal, rows=200)


def test_growing_and_large_scores(cuda_lib):
    import torch
    n = 900
    q, k, v = _inputs(n, 4, 1, 128, "bf16", 8, fused=False)
    q[:] = q[0, 0]
    k[:, 0] = (torch.linspace(0.01, 4.0, n, device="cuda")[:, None] * q[0, 0].float()).to(k.dtype)
    for scale in (128 ** -0.5, -128 ** -0.5, 0.0):
        _check(cuda_lib, q, k, v, [0, n], "bf16", True, rows=60, scale=scale)
        _check(cuda_lib, q, k, v, [0, 400, n], "bf16", False, rows=60, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (5, 1)])
def test_infinities_and_nan_reach_only_rows_that_see_them(cuda_lib, dtype, bad, Hq, Hkv):
    import torch
    lens, G = [150, 90, 300], Hq // Hkv
    cu = _cu(lens)
    q, k, v = _inputs(sum(lens), Hq, Hkv, 128, dtype, 9, fused=False)
    clean, clean_lse = _run(cuda_lib, q, k, v, cu)
    full, full_lse = _run(cuda_lib, q, k, v, cu, causal=False)
    t = 200                                        # in the second sequence, [150, 240)
    v[t, 0, 5] = bad
    out, lse = _run(cuda_lib, q, k, v, cu)
    assert torch.equal(out[:t], clean[:t]) and torch.equal(out[240:], clean[240:])
    assert torch.equal(out[:, G:], clean[:, G:]) and torch.equal(lse, clean_lse)
    hit = out[t:240, :G, 5].float()
    assert bool(hit.isnan().all()) if math.isnan(bad) else bool((hit == bad).all())
    rest = [d for d in range(128) if d != 5]
    tol = 4 * ULP[dtype] * 5
    assert float((out[..., rest].float() - clean[..., rest].float()).abs().max()) <= tol
    out, _ = _run(cuda_lib, q, k, v, cu, causal=False)
    assert torch.equal(out[:150], full[:150]) and torch.equal(out[240:], full[240:])
    hit = out[150:240, :G, 5].float()
    assert bool(hit.isnan().all()) if math.isnan(bad) else bool((hit == bad).all())
    v[t, 0, 5] = 0.0
    k[t, 0] = bad
    out, lse = _run(cuda_lib, q, k, v, cu)
    assert torch.equal(out[:t], clean[:t]) and torch.equal(out[240:], clean[240:])


def test_repeats_streams_and_graphs(cuda_lib):
    import torch
    lens = [700, 33, 1200]
    q, k, v = _inputs(sum(lens), 8, 2, 128, "bf16", 10)
    ws = cuda_lib.Workspace(cuda_lib.OP_PROMPT_ATTENTION, 3, sum(lens), 8, 128)
    ws.buf.fill_(255)
    a, la = _run(cuda_lib, q, k, v, _cu(lens), workspace=ws)
    cu = torch.tensor(_cu(lens), dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(a), torch.empty_like(la)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cuda_lib.dspark_prompt_attention(q, k, v, cu, 128 ** -0.5, out=out, lse=lse, workspace=ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(la, lse)
    assert cuda_lib.dspark_read_status(ws) == (0, 0)


def test_bounds_out_of_order_are_flagged(cuda_lib):
    import torch
    q, k, v = _inputs(200, 4, 2, 64, "bf16", 12)
    ws = cuda_lib.Workspace(cuda_lib.OP_PROMPT_ATTENTION, 4, 200, 4, 64)
    out, lse = _run(cuda_lib, q, k, v, [-5, 60, 30, 120, 1000], workspace=ws)
    assert cuda_lib.dspark_read_status(ws)[1] & cuda_lib.STATUS_INPUT_RANGE
    good, good_lse = _run(cuda_lib, q, k, v, [0, 60, 60, 120, 200], workspace=ws)
    assert cuda_lib.dspark_read_status(ws) == (0, 0)
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    q, k, v = _inputs(20, 4, 2, 64, "bf16", 13)
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        ds.dspark_prompt_attention(q.float(), k, v, cu, 0.1)
    with pytest.raises(TypeError):
        ds.dspark_prompt_attention(q, k, v.half(), cu, 0.1)
    with pytest.raises(TypeError):
        ds.dspark_prompt_attention(q, k, v, cu.long(), 0.1)
    with pytest.raises(ValueError):
        ds.dspark_prompt_attention(q.transpose(0, 1), k, v, cu, 0.1)
    with pytest.raises(ValueError):
        ds.dspark_prompt_attention(q, k[:10], v[:10], cu, 0.1)
    with pytest.raises(ValueError):
        ds.dspark_prompt_attention(q, k, v, cu, 0.1, lse=torch.empty(20, 5, device="cuda"))
    odd = torch.zeros(20, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :256].view(20, 4, 64)
    for args, kw in (((q[:, :3], k, v, cu, 0.1), {}), ((q, k, v, cu, math.nan), {}), ((q, k, v, cu[:1], 0.1), {}),
                     ((odd, k, v, cu, 0.1), {})):
        with pytest.raises(ds.DSparkError) as e:
            ds.dspark_prompt_attention(*args, **kw)
        assert e.value.status == 1
