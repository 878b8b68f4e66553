"""GPU parity of the tree operators where their sizes end: rows around one and two tiles with and without lengths, windows
past 32 bits, the largest vocabulary, many small requests, a workspace that calls of all kinds share."""
import math

import numpy as np
import pytest

from tests._trees import WindowCase
from tests.test_gpu_tree_attention import _tree
from tests.test_gpu_verify_tree import VerifyCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,N", [(4, 31), (4, 32), (4, 33), (4, 63), (4, 64), (4, 65), (3, 42), (3, 43), (3, 84), (3, 85), (128, 1),
                                 (128, 2), (128, 3), (65, 2), (65, 3), (1, 256)])
def test_rows_around_one_and_two_tiles(cuda_lib, D, G, N):
    rng = np.random.default_rng(N + G)
    lens = [N, N + 1, N + 128, 700, 0, 2000]
    lengths = [N, max(0, N - 1), N // 2, 1, 0, N]
    case = _tree(len(lens), N, G * 2, 2, D, 16, lens, seed=N * 10 + G)
    window = WindowCase(len(lens), N, G * 2, 2, D, 16, lens, seed=N * 10 + G + 1, window=90, sinks=int(rng.integers(0, 5)))
    for ln in (lengths, [min(N, x) for x in lens]):
        case.check(cuda_lib, lengths=ln, rows=100)
        window.check(cuda_lib, lengths=ln, rows=100)
        window.check(cuda_lib, lengths=ln, causal=False, rows=100)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("N", [33, 64, 65, 150])
def test_infinities_in_requests_with_lengths(cuda_lib, bad, N):
    """A value that only some rows of some tiles see, one request of three."""
    import torch
    lens = [400, 300, 131 + N]
    lengths = [N, N - 20, 7]
    case = _tree(3, N, 8, 2, 128, 16, lens, seed=13)
    case.parents[0, :5] = [-1, 0, 0, 1, 2]
    clean, clean_lse = case.run(cuda_lib, lengths=lengths)
    j = lens[0] - N + 1                                       # node 1's
    at = (int(case.table[0, j // 16]), 1, j % 16)
    case.v[at][5] = bad
    out, lse = case.run(cuda_lib, lengths=lengths)
    hit = torch.tensor([j in case.sees(0, i, lengths, True) for i in range(N)], device="cuda")
    assert bool(hit[1]) and bool(hit[3]) and not bool(hit[[0, 2, 4]].any())
    assert torch.equal(out[0, ~hit], clean[0, ~hit]) and torch.equal(lse, clean_lse)
    assert torch.equal(out[1:], clean[1:]) and torch.equal(out[0, :, :4], clean[0, :, :4])
    got = out[0, hit][:, 4:, 5].float()
    assert bool(got.isnan().all()) if math.isnan(bad) else bool((got == bad).all())


@pytest.mark.parametrize("window,sinks,like", [(2 ** 32 + 5, 0, (2 ** 31 - 1, 0)), (2 ** 70, 2 ** 32, (2 ** 31 - 1, 2 ** 31 - 1)),
                                               (20, 2 ** 32 + 1, (20, 2 ** 31 - 1))])
def test_numbers_past_32_bits_are_not_cut(cuda_lib, window, sinks, like):
    import torch
    case = WindowCase(2, 9, 4, 2, 64, 16, [300, 90], seed=5, window=window, sinks=sinks)
    tree = _tree(2, 9, 4, 2, 64, 16, [300, 90], seed=5, window=window, sinks=sinks)
    for c in (case, tree):
        got, _ = c.run(cuda_lib)
        c.window, c.sinks = like
        want, _ = c.run(cuda_lib)
        assert torch.equal(got, want)
        c.window = -2 ** 32 + 20                              # below what a C int holds: refused, not read as 20
        with pytest.raises(cuda_lib.DSparkError) as e:
            c.run(cuda_lib)
        assert e.value.status == 1


@pytest.mark.parametrize("bf16", [False, True])
def test_the_largest_vocabulary(cuda_lib, bf16):
    VerifyCase(2, 5, 1 << 21, seed=3, bf16=bf16, follow=1.0).check(cuda_lib)
    VerifyCase(40, 2, (1 << 21) - 3, seed=4, bf16=bf16, follow=1.0).check(cuda_lib)


def test_many_small_requests(cuda_lib):
    VerifyCase(3000, 2, 5, seed=6, lengths=np.arange(3000) % 3).check(cuda_lib)


def test_one_workspace_for_calls_in_turn(cuda_lib):
    """Larger and smaller calls of both attentions and both kernels, one after the other, on one workspace."""
    import torch
    ds = cuda_lib
    ws = ds.Workspace(ds.OP_TREE_ATTENTION, 3, 200, 8, 128)
    cases = [_tree(3, 200, 8, 2, 128, 16, [900, 300, 5000], seed=1), _tree(2, 20, 8, 2, 64, 16, [900, 3000], seed=2),
             WindowCase(3, 64, 8, 2, 128, 16, [900, 300, 64], seed=3, window=70, sinks=1)]
    lengths = ([200, 100, 3], [20, 1], [64, 0, 33])
    want = [(c.run(ds), c.run(ds, lengths=ln)) for c, ln in zip(cases, lengths)]
    for _ in range(3):
        for c, ln, (full, part) in zip(cases, lengths, want):
            a, b = c.run(ds, workspace=ws), c.run(ds, lengths=ln, workspace=ws)
            for x, y in ((a, full), (b, part)):
                assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert ds.dspark_read_status(ws) == (0, 0)
