"""The serving example: the operators together against a plain recomputation in 64 bits.

Every target pass of a served batch is recomputed from the requests' tokens alone: no cache, no
pages, no windows.  The recomputation follows the model's roundings to bf16 (projections, rotated
queries and keys, attention output, hidden state), so what is left is the order of sums and the
few rounding choices that they tip.
"""
import math

import pytest
import torch

from examples import serving_round as ex

pytestmark = pytest.mark.gpu


def _bf16(x):
    return x.to(torch.bfloat16).double()


def _plain_logits(shape, w, tokens):
    """Logits [T, V] of one request's tokens, in 64 bits with the model's roundings."""
    w = {k: v.double().cpu() for k, v in w.items()}
    T = len(tokens)
    x = w["embed"][torch.tensor(tokens)]
    qkv = _bf16(x @ w["qkv"])
    q, k, v = (t.unflatten(1, (-1, shape.D)) for t in
               qkv.split([shape.Hq * shape.D, shape.Hkv * shape.D, shape.Hkv * shape.D], 1))
    table = ex.rotation_table(shape, "cpu").double()[:T]
    cos, sin = table[:, None, :shape.D // 2], table[:, None, shape.D // 2:]

    def turned(t):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        a, b = t[..., :shape.D // 2], t[..., shape.D // 2:]
        return _bf16(torch.cat([a * cos - b * sin, b * cos + a * sin], -1))

    q, k = turned(q), turned(k)
    g = shape.Hq // shape.Hkv
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("ihd,jhd->hij", q, k) * shape.D ** -0.5
    s = s.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
    o = _bf16(torch.einsum("hij,jhd->ihd", s.softmax(-1), v)).flatten(1)
    h = _bf16(x + _bf16(o @ w["out"]))
    return h @ w["lm_head"].T


# A hidden value of size up to about 5 moves by at most one or two of its bf16 spacings (2^-8 relative) when a
# rounding is tipped; few of the 512 are.  A logit is their sum with weights of 3 / sqrt(512): all 512 tipped at
# random would move it by 3 * 5 * 2^-8 = 0.06 in the root mean square, five of which no logit exceeds.
LOGIT_BOUND = 0.3


@pytest.mark.parametrize("greedy", [True, False])
def test_served_batch_matches_plain_recomputation(cuda_lib, greedy):
    shape = ex.Shape(V=1024, H=512)
    dev = torch.device("cuda:0")
    weights = ex.random_weights(shape, 3, dev)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(shape.V, (n,), generator=g).tolist() for n in (1, 130, 16, 37)]
    B, gamma, rounds = len(prompts), 3, 4
    full = lambda x, dtype=torch.float32: torch.full((B,), x, dtype=dtype, device=dev)
    sampling = ex.Sampling(full(1.0), full(1 if greedy else 40, torch.int32), full(1.0 if greedy else 0.9), full(0.0))
    passes = []

    def trace(text, first, window, logits):
        passes.append(([list(t) for t in text], first, None if window is None else window.tolist(), logits.double().cpu()))

    text, accepted = ex.serve(shape, weights, ex.perturbed(weights, 0.02, 5), prompts, sampling, gamma, rounds, 7, trace)
    assert len(passes) == rounds + 1 and 0.0 <= accepted <= gamma
    for before, first, window, logits in passes:
        row = 0
        for b in range(B):
            if window is None:
                tokens, n = before[b], len(before[b])
            else:
                assert before[b][first[b]:] == window[b][:1]
                tokens, n = before[b][:first[b]] + window[b], gamma + 1
            plain = _plain_logits(shape, weights, tokens)[-n:]
            assert (logits[row:row + n] - plain).abs().max() < LOGIT_BOUND
            row += n
    for p, t in zip(prompts, text):
        assert t[:len(p)] == p and len(t) >= len(p) + 1 + rounds
        plain = _plain_logits(shape, weights, t[:-1])
        for i in range(len(p), len(t)):
            row = plain[i - 1]
            if greedy:                                                   # the largest logit, but for near ties
                assert row.max() - row[t[i]] < 2 * LOGIT_BOUND
            else:                                                        # among the 40 largest
                assert row[t[i]] > row.topk(40).values[-1] - 2 * LOGIT_BOUND
