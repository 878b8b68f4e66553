"""GPU parity where the serving operators' launches take another path by size alone: more rows than SMs that are too
long to be held in shared memory, more prompts than are put in order of their work, more requests than one scan of
the plan takes, and windows of several row tiles."""
import numpy as np
import pytest

from tests._serving import PagedCase
from tests.test_gpu_prompt_attention import _check, _cu, _inputs
from tests.test_gpu_sample import Rows, _normal, _settings
from tests.test_gpu_sample_ties import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,V,bf16", [(170, 60001, False), (170, 110001, True), (153, 151936, False)])
def test_sampling_long_rows_from_the_queue(cuda_lib, R, V, bf16):
    import torch
    rng = np.random.default_rng(V)
    check(cuda_lib, Rows(_normal(R, V, V, dtype=torch.bfloat16 if bf16 else None), *_settings(rng, R)), oracle_rows=4)


@pytest.mark.parametrize("R", [151, 152, 153, 305])
def test_sampling_around_a_row_per_block(cuda_lib, R):
    rng = np.random.default_rng(R)
    check(cuda_lib, Rows(_normal(R, 20011, R), *_settings(rng, R)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,longest", [(256, 60), (257, 60), (300, 900), (1100, 40), (2100, 5)])
def test_many_prompts_some_of_them_empty(cuda_lib, B, longest, causal):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, longest + 1, B)
    lens[rng.random(B) < 0.2] = 0
    if longest > 500:
        lens[rng.random(B) < 0.8] //= 20
    cu = [int(x) + 2 for x in _cu(lens.tolist())]                          # two tokens ahead of the first
    q, k, v = _inputs(cu[-1] + 3, 4, 2, 64, "bf16", B)
    out, _ = _check(cuda_lib, q, k, v, cu, "bf16", causal, rows=300)
    assert not out[:2].any() and not out[-3:].any()


@pytest.mark.parametrize("B", [1024, 1025, 2500])
def test_many_requests(cuda_lib, B):
    rng = np.random.default_rng(B)
    lens = np.exp(rng.uniform(0, np.log(300), B)).astype(int)
    lens[rng.random(B) < 0.1] = 0
    lengths = np.minimum(rng.integers(0, 4, B), lens)
    case = PagedCase(B, 3, 4, 2, 64, 16, lens.tolist(), seed=B)
    for causal in (True, False):
        out, lse = case.check(cuda_lib, lengths=lengths.tolist(), causal=causal, rows=300)
        assert not out[lengths == 0].any() and bool((lse[lengths == 0] == -np.inf).all())


def test_many_requests_with_long_ones_behind(cuda_lib):
    lens = [1] * 1500 + [9000, 0, 3001] + [2] * 600 + [5000]
    case = PagedCase(len(lens), 1, 4, 1, 128, 64, lens, seed=3)
    out, lse = case.check(cuda_lib, rows=100)
    for b in (1500, 1502, len(lens) - 1):
        for h in range(4):
            ref = case.row(b, 0, h)
            np.testing.assert_allclose(lse[b, 0, h].item(), ref[1], atol=1e-3)
            np.testing.assert_allclose(out[b, 0, h].float().cpu().numpy(), ref[0], atol=0.02)


@pytest.mark.parametrize("N,G,D,dtype", [(257, 2, 64, "bf16"), (300, 4, 128, "f16"), (1000, 1, 128, "bf16"), (130, 7, 64, "f16")])
def test_long_windows_over_a_prefix(cuda_lib, N, G, D, dtype):
    lens = [N, N + 700, N + 1, 3 * N + 5]
    lengths = [N, N - 3, 1, N]
    case = PagedCase(len(lens), N, 2 * G, 2, D, 32, lens, dtype, seed=N)
    for causal in (True, False):
        case.check(cuda_lib, lengths=lengths, causal=causal, rows=250)


def test_prompt_offsets_past_32_bits(cuda_lib):
    """Queries and outputs of more than 2^31 values: the last sequence as in a call of its own."""
    import torch
    Hq, D, n, B = 128, 128, 70, 2000
    T = B * n
    assert T * Hq * D > 1 << 31
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = _inputs(n, Hq, 1, D, "bf16", 1, fused=False)
    for whole, part in zip((q, k, v), small):
        whole[-n:] = part
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    lse, want_lse = torch.empty(T, Hq, device="cuda"), torch.empty(n, Hq, device="cuda")
    out = cuda_lib.dspark_prompt_attention(q, k, v, cu, D ** -0.5, lse=lse)
    want = cuda_lib.dspark_prompt_attention(*small, cu[:2].contiguous(), D ** -0.5, lse=want_lse)
    assert torch.equal(out[-n:], want) and torch.equal(lse[-n:], want_lse)
    assert not out[:-n].any()


def test_sampling_offsets_past_32_bits(cuda_lib):
    """More than 2^31 logits and probabilities: the last rows as in a call of their own."""
    import torch
    R, V, last = 14200, 151936, 20
    assert R * V > 1 << 31
    rng = np.random.default_rng(5)
    small = Rows(_normal(last, V, 5), *_settings(rng, last))
    want, want_probs = small.run(cuda_lib)
    big = Rows(torch.zeros(R, V, device="cuda"), np.zeros(R), np.zeros(R, int), np.ones(R), np.zeros(R), np.zeros(R))
    for name in ("logits", "T", "k", "p", "mp", "u"):
        getattr(big, name)[-last:] = getattr(small, name)
    tok, probs = big.run(cuda_lib)
    assert torch.equal(tok[-last:], want) and torch.equal(probs[-last:], want_probs)
    assert not tok[:-last].any() and bool((probs[:-last, 0] == 1).all())
