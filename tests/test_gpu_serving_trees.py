"""The serving example with trees: the operators together against a plain recomputation in 64 bits.

Every node that the target scores is recomputed from its sequence's tokens and its path in the tree alone: no cache, no
pages, no trees, no moves.  What the last rounds accepted and moved is in the sequences that the next ones are
recomputed from, so a key or value in a wrong place shows.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from examples import serving_round as ex
from tests.test_gpu_serving_round import LOGIT_BOUND, _bf16

pytestmark = pytest.mark.gpu


def _plain_logits(shape, w, tokens):
    """Logits [V] behind the last of one sequence's tokens, in 64 bits with the model's roundings."""
    w = {k: v.double().cpu() for k, v in w.items()}
    T = len(tokens)
    x = w["embed"][torch.tensor(tokens)]
    q, k, v = (t.unflatten(1, (-1, shape.D)) for t in
               _bf16(x @ w["qkv"]).split([shape.Hq * shape.D, shape.Hkv * shape.D, shape.Hkv * shape.D], 1))
    table = ex.rotation_table(shape, "cpu").double()[:T]
    cos, sin = table[:, None, :shape.D // 2], table[:, None, shape.D // 2:]

    def turned(t):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        a, b = t[..., :shape.D // 2], t[..., shape.D // 2:]
        return _bf16(torch.cat([a * cos - b * sin, b * cos + a * sin], -1))

    q, k = turned(q)[-1], turned(k)
    g = shape.Hq // shape.Hkv
    s = torch.einsum("hd,jhd->hj", q, k.repeat_interleave(g, 1)) * shape.D ** -0.5
    if shape.window:
        j = torch.arange(T)
        s = s.masked_fill((j >= shape.sinks) & (j <= T - 1 - shape.window), -math.inf)
    o = _bf16(torch.einsum("hj,jhd->hd", s.softmax(-1), v.repeat_interleave(g, 1))).flatten()
    return _bf16(x[-1] + _bf16(o @ w["out"])) @ w["lm_head"].T


def _path(parents, i):
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out[::-1]


@pytest.mark.parametrize("mode", ["greedy", "temperature", "sampling"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_trees_match_plain_recomputation(cuda_lib, mode, window, sinks):
    shape = ex.Shape(V=1024, H=512, window=window, sinks=sinks)
    dev = torch.device("cuda:0")
    weights = ex.random_weights(shape, 3, dev)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(shape.V, (n,), generator=g).tolist() for n in (1, 130, 16, 37)]
    samples, branching = 2, [3, 2, 1]
    B = len(prompts) * samples
    rng = np.random.default_rng(0)
    full = lambda x, t=torch.float32: torch.full((B,), x, dtype=t, device=dev)
    sampling = ex.Sampling(full(0.9), full(20, torch.int32), full(0.9), full(0.0)) if mode == "sampling" else None
    seen = []

    def trace(text, tokens, tree, logits, decision):
        N = tokens.shape[1]
        tokens, parents, logits = tokens.cpu(), tree[0].tolist(), logits.view(B, N, -1).double().cpu()
        out, accepted, path = (t.cpu() for t in decision)
        assert (tokens[:, 0] == torch.tensor([t[-1] for t in text])).all()
        for b in range(B):
            for i in rng.choice(N, 3, replace=False).tolist() + [int(path[b, int(accepted[b])])]:
                line = text[b][:-1] + [int(tokens[b, x]) for x in _path(parents, i)]
                err = float((_plain_logits(shape, weights, line) - logits[b, i]).abs().max())
                assert err <= LOGIT_BOUND, (b, i, err)
            n = int(accepted[b])
            for x, y in zip(path[b, :n].tolist(), path[b, 1:n + 1].tolist()):
                assert parents[y] == x
            assert out[b, :n].tolist() == [int(tokens[b, x]) for x in path[b, 1:n + 1].tolist()]
            if mode == "greedy":
                want, nodes = oracle.verify_tree(lambda i: int(logits[b, i].argmax()), parents, tokens[b].tolist(), N)
                assert out[b, :n + 1].tolist() == want and path[b, :n + 1].tolist() == nodes
        seen.append(int(accepted.sum()))

    text, accepted = ex.serve_trees(shape, weights, ex.perturbed(weights, 0.02, 5), prompts, branching, 5, samples,
                                    temperature=0.0 if mode == "greedy" else 0.9, sampling=sampling, seed=6, chunk=64, trace=trace)
    assert len(seen) == 5 and sum(seen) > 0 and accepted == sum(seen) / (B * 5)
    for i, t in enumerate(text):
        p = prompts[i // samples]
        assert t[:len(p)] == p and len(t) >= len(p) + 1 + 5
