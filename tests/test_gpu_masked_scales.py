"""GPU parity of the masked attentions at scales of every sign and size, in every kernel that serves them.

Rows of a key head: 1 and 8 (four copies of the rows in a tile), 48 (two), 124 (one), 256 and 600 (two row tiles to a unit;
with lengths, 256 take one).  Keys that grow along the request make the running maximum rise from tile to tile; scales below
zero turn the order of the products around; at a scale of 0, or one that fp32 holds in few bits, a masked score must still get
no weight.
"""
import numpy as np
import pytest

from tests._serving import PagedCase, attention_tolerance, check_attention, lse_tolerance
from tests._trees import TreeCase, WindowCase, random_parents

pytestmark = pytest.mark.gpu

ROWS = [(1, 1), (2, 4), (12, 4), (31, 4), (64, 4), (150, 4)]


def _grow(case, sign):
    """Keys along the first row's query of their head, longer and longer."""
    import torch
    for b in range(len(case.kv_len)):
        j = np.arange(case.kv_len[b])
        ramp = torch.linspace(0.01, 4.0, len(j), device="cuda")[:, None, None] * case.q[b, 0, ::case.group].float()
        case.k[case.table[b, j // case.page], :, j % case.page] = (sign * ramp).to(case.k.dtype)


def _scales(case, ds, causals, lengths):
    plain = case.scale
    for ln in (None, lengths):
        for causal in causals:
            _grow(case, 1.0)
            for scale in (plain, -plain, 0.0, 1e-40, -1e-40):
                case.scale = scale
                case.check(ds, lengths=ln, causal=causal, rows=24)
            _grow(case, -1.0)
            case.scale = -plain
            case.check(ds, lengths=ln, causal=causal, rows=24)
            case.scale = plain


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", ROWS)
def test_windows(cuda_lib, dtype, D, N, G):
    case = WindowCase(2, N, 2 * G, 2, D, 16, [900, 700], dtype, seed=N, window=400, sinks=9)
    _scales(case, cuda_lib, (True, False), [N, max(1, N - 3)])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", ROWS)
def test_trees(cuda_lib, dtype, D, N, G):
    parents = random_parents(np.random.default_rng(N), 2, N, deepest=9)
    case = TreeCase(2, N, 2 * G, 2, D, 16, [900, 700], dtype, seed=N, parents=parents)
    _scales(case, cuda_lib, (True,), [N, max(1, N - 3)])
    case.window, case.sinks = N + 200, 9
    _scales(case, cuda_lib, (True,), [N, max(1, N - 3)])


def _dense(case, b, n, causal):
    """Every row of a request in 64 bits, without a window: (out, lse, spread, size), [n, Hq, ...]."""
    import torch
    L = int(case.kv_len[b])
    j = np.arange(L)
    K, V = (t[case.table[b, j // case.page], :, j % case.page].double().repeat_interleave(case.group, 1) for t in (case.k, case.v))
    q = case.q[b, :n].double()
    s = torch.einsum("nhd,lhd->nhl", q, K) * case.scale
    size = torch.einsum("nhd,lhd->nhl", q.abs(), K.abs()) * abs(case.scale)
    if causal:
        hidden = torch.arange(L, device="cuda")[None, :] > (L - n + torch.arange(n, device="cuda"))[:, None]
        s, size = s.masked_fill(hidden[:, None], -float("inf")), size.masked_fill(hidden[:, None], 0.0)
    p = torch.softmax(s, dim=2)
    return [x.cpu().numpy() for x in (torch.einsum("nhl,lhd->nhd", p, V), s.logsumexp(2), torch.einsum("nhl,lhd->nhd", p, V.abs()), size.amax(2))]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N", [1, 17, 33, 70, 150])
def test_a_window_wider_than_the_cache_equals_none(cuda_lib, N, dtype):
    """Every row.  Two kernels that are each within the tolerance of the exact value differ by at most twice that."""
    import torch
    lens = [max(L, N) for L in (40, 150, 300, 1000, 129)]
    case = WindowCase(5, N, 8, 2, 128, 16, lens, dtype, seed=3, window=1100, sinks=0)
    plain = PagedCase(5, N, 8, 2, 128, 16, lens, dtype, seed=3)
    for lengths in (None, [N, max(1, N // 5), 0, N, max(1, N // 2)]):
        for causal in (True, False):
            a, la = case.run(cuda_lib, lengths=lengths, causal=causal)
            b, lb = plain.run(cuda_lib, lengths=lengths, causal=causal)
            for r in range(5):
                n = N if lengths is None else lengths[r]
                assert not a[r, n:].any() and not b[r, n:].any() and torch.equal(la[r, n:], lb[r, n:])
                if n == 0:
                    continue
                ref = _dense(case, r, n, causal)
                check_attention(a[r, :n], la[r, :n], ref, dtype, lens[r], 6.0)
                out, lse, spread, size = ref
                far = (a[r, :n].double() - b[r, :n].double()).abs().cpu().numpy()
                assert (far <= 2 * attention_tolerance(out, spread, size, dtype, lens[r], 6.0)).all()
                assert ((la[r, :n].double() - lb[r, :n].double()).abs().cpu().numpy() <= 2 * lse_tolerance(lse, size)).all()
