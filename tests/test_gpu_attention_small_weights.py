"""GPU parity: fp16 attention whose mass lies in many weights far below the row's largest.

One key takes nearly all the weight (an attention sink, whose value is zero here, so that the output is
what the others bring), and the others have weights around 2^-25 of it, or over a wide range below it.
The weights of the product with v are at most 2^15 and rounded to fp16, so a weight of 2^-25 of the
largest is 2^-18 or more: its rounding is at most 2^-25, which is 2^-32 of the largest.
"""
import math

import numpy as np
import pytest

import oracle
from tests._serving import PagedCase, check_attention, f64

pytestmark = pytest.mark.gpu
SCALE = 0.125                                               # with q = 8 in one place, a key's value there is its score


def _scores(n, kind, seed):
    """A sink of score 0 among n keys, and where it is."""
    rng = np.random.default_rng(seed)
    if kind == "just_below":
        s = np.full(n, -25.1 * math.log(2.0))
    elif kind == "range":
        s = -math.log(2.0) * rng.uniform(12.0, 31.0, n)
    else:                                                   # the largest is reached by steps below 2^8, never raised
        s = np.linspace(-5.4, -4.0, n) - math.log(2.0) * rng.uniform(0.0, 20.0, n)
    at = n - 1 if kind == "steps" else min(3, n - 1)
    s[at] = 0.0
    if kind == "steps":
        s[:2] = -5.4
    return s, at


def _check(out, lse, ref, keys):
    # tests/_serving.py's bound with its term for weights rounded to a fixed step 2^7 smaller
    check_attention(out, lse, ref, "f16", keys / 128.0, 1.5)


@pytest.mark.parametrize("kind", ["just_below", "range", "steps"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G,L", [(1, 1, 131072), (1, 4, 300), (5, 8, 20001), (17, 5, 5000), (17, 5, 131)])
def test_paged(cuda_lib, kind, D, N, G, L):
    import torch
    case = PagedCase(1, N, G, 1, D, 64, [L], "f16", seed=L + N)
    case.scale = SCALE
    s, at = _scores(L - N + 1, kind, L)
    s = np.concatenate([s, np.full(N - 1, s.min())])        # the window's own tokens
    j = np.arange(L)
    pages, offs = case.table[0, j // 64], j % 64
    key = torch.zeros(L, D, device="cuda")
    key[:, 0] = torch.from_numpy(s).cuda()
    case.k[pages, 0, offs] = key.half()
    case.v[pages, 0, offs] = (0.5 + torch.rand(L, D, generator=torch.Generator(device="cuda").manual_seed(L), device="cuda")).half()
    case.v[int(pages[at]), 0, int(offs[at])] = 0.0
    case.q.zero_()
    case.q[..., 0] = 8.0
    out, lse = case.run(cuda_lib)
    rows = [(0, i, h) for i in sorted({0, N // 2, N - 1}) for h in sorted({0, G - 1})]
    ref = [np.array(x) for x in zip(*(case.row(*r) for r in rows))]
    idx = tuple(torch.tensor(x, device="cuda") for x in zip(*rows))
    _check(out[idx], lse[idx], ref, L)


@pytest.mark.parametrize("kind", ["just_below", "range", "steps"])
def test_paged_long_context_in_one_piece(cuda_lib, kind):
    """More requests than SMs over the same pages: most are not cut, and sum all their keys in one place."""
    import torch
    B, L, D = 160, 131072, 64
    case = PagedCase(1, 1, 1, 1, D, 64, [L], "f16", seed=7)
    case.scale = SCALE
    s, at = _scores(L, kind, 7)
    j = np.arange(L)
    pages, offs = case.table[0, j // 64], j % 64
    case.k[pages, 0, offs] = torch.nn.functional.pad(torch.from_numpy(s).cuda()[:, None], (0, D - 1)).half()
    case.v[pages, 0, offs] = (0.5 + torch.rand(L, D, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")).half()
    case.v[int(pages[at]), 0, int(offs[at])] = 0.0
    case.q = torch.zeros(B, 1, 1, D, device="cuda", dtype=torch.float16)
    case.q[..., 0] = 8.0
    case.table, case.kv_len = np.repeat(case.table, B, 0), np.repeat(case.kv_len, B)
    out, lse = case.run(cuda_lib)
    ref = [np.array(x)[None] for x in case.row(0, 0, 0)]
    for b in (0, 1, 70, 159):
        _check(out[b, 0], lse[b, 0], ref, L)


@pytest.mark.parametrize("kind", ["just_below", "range", "steps"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,T", [(1, 2000), (4, 700), (5, 130)])
def test_prompt(cuda_lib, kind, D, causal, G, T):
    import torch
    s, at = _scores(T, kind, T)
    if causal and kind == "steps":                          # the sink where most rows see it
        s[[at, T // 3]] = s[[T // 3, at]]
        at = T // 3
    q = torch.zeros(T, G, D, device="cuda", dtype=torch.float16)
    q[..., 0] = 8.0
    k = torch.zeros(T, 1, D, device="cuda", dtype=torch.float16)
    k[:, 0, 0] = torch.from_numpy(s).cuda().half()
    v = (0.5 + torch.rand(T, 1, D, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")).half()
    v[at] = 0.0
    lse = torch.empty(T, G, device="cuda")
    out = cuda_lib.dspark_prompt_attention(q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), SCALE, causal=causal,
                                           lse=lse)
    rows = [(t, h) for t in sorted({0, 5, T // 2, T - 2, T - 1}) for h in sorted({0, G - 1})]
    ref = []
    for t, h in rows:
        end = t + 1 if causal else T
        ref.append(oracle.attend_row(f64(q[t, h]), f64(k[:end, 0]), f64(v[:end, 0]), SCALE))
    idx = tuple(torch.tensor(x, device="cuda") for x in zip(*rows))
    _check(out[idx], lse[idx], [np.array(x) for x in zip(*ref)], T)
