"""Speculative serving of a few requests on one GPU, with the library's serving operators together.

A one-layer attention model with random weights is served to a batch of requests:

    prompts     dspark_kv_append (rotation, cache) + dspark_prompt_attention
    drafting    gamma single-token steps of a perturbed copy of the model: dspark_kv_append,
                dspark_paged_attention, dspark_draft_logits, dspark_sample (with distributions)
    verifying   one window of gamma + 1 tokens per request through the model: the same calls, then
                dspark_verify on the two sides' truncated distributions

Run it on a GB300 after building the library:  python examples/serving_round.py
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import draft_sampling_verification_tcgen05_gb300 as ds


@dataclass
class Shape:
    V: int = 4096          # vocabulary
    H: int = 512           # hidden size
    Hq: int = 8
    Hkv: int = 2
    D: int = 64
    page: int = 16
    max_positions: int = 2048


def rotation_table(shape: Shape, device) -> torch.Tensor:
    """[max_positions, D] fp32: the cosines of D / 2 angles, then their sines."""
    freq = 10000.0 ** (-torch.arange(0, shape.D, 2, dtype=torch.float64) / shape.D)
    angle = torch.arange(shape.max_positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device).contiguous()


class Model:
    """Weights of one attention layer and the calls that run it."""

    def __init__(self, shape: Shape, weights: dict, num_pages: int):
        self.shape, self.w = shape, weights
        dev = weights["embed"].device
        s = shape
        self.table = rotation_table(s, dev)
        self.k_cache = torch.zeros(num_pages, s.Hkv, s.page, s.D, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.scale = s.D ** -0.5
        self.workspaces: dict = {}

    def _workspace(self, op, *sizes):
        key = (op,) + sizes
        if key not in self.workspaces:
            self.workspaces[key] = ds.Workspace(op, *sizes)
        return self.workspaces[key]

    def append(self, tokens, positions, slots):
        """Caches the tokens' keys and values; returns (hidden [T, H], rotated q, k, v)."""
        s = self.shape
        x = self.w["embed"][tokens.long()]
        qkv = x @ self.w["qkv"]
        q, k, v = (t.unflatten(1, (-1, s.D)) for t in qkv.split([s.Hq * s.D, s.Hkv * s.D, s.Hkv * s.D], 1))
        q = ds.dspark_kv_append(q, k, v, positions, slots, self.table, self.k_cache, self.v_cache,
                                q_norm=self.w["q_norm"], k_norm=self.w["k_norm"],
                                workspace=self._workspace(ds.OP_KV_APPEND))
        return x, q, k, v

    def logits(self, x, attended):
        h = x + attended.flatten(1) @ self.w["out"]
        return ds.dspark_draft_logits(h, self.w["lm_head"], workspace=self._workspace(ds.OP_DRAFT_LOGITS))

    def prompt(self, tokens, positions, slots, cu_seqlens):
        """All prompts, packed; returns the logits of every token."""
        s = self.shape
        x, q, _, v = self.append(tokens, positions, slots)
        k = self.gather_keys(slots)
        ws = self._workspace(ds.OP_PROMPT_ATTENTION, cu_seqlens.shape[0] - 1, q.shape[0], s.Hq, s.D)
        return self.logits(x, ds.dspark_prompt_attention(q, k, v, cu_seqlens, self.scale, workspace=ws))

    def gather_keys(self, slots):
        """The rotated keys as the cache holds them, [T, Hkv, D]."""
        page = self.shape.page
        return self.k_cache[(slots // page).long(), :, (slots % page).long()].contiguous()

    def window(self, tokens, positions, slots, block_table, kv_len):
        """A window of N tokens per request, tokens [B, N]; returns logits [B * N, V]."""
        s = self.shape
        B, N = tokens.shape
        x, q, _, _ = self.append(*(t.flatten().contiguous() for t in (tokens, positions, slots)))
        ws = self._workspace(ds.OP_PAGED_ATTENTION, B, N, s.Hq, s.D)
        o = ds.dspark_paged_attention(q.view(B, N, s.Hq, s.D), self.k_cache, self.v_cache, block_table, kv_len,
                                      self.scale, workspace=ws)
        return self.logits(x, o.view(B * N, s.Hq, s.D))


class Sampling:
    """The requests' sampling parameters, a row per request and window token."""

    def __init__(self, temperature, top_k, top_p, min_p):
        self.columns = (temperature, top_k, top_p, min_p)

    def __call__(self, logits, u):
        """Tokens [R] and their truncated distributions [R, V]; R a multiple of the requests."""
        n = logits.shape[0] // self.columns[0].shape[0]
        probs = torch.empty_like(logits)
        tokens = ds.dspark_sample(logits, *(c.repeat_interleave(n) for c in self.columns), u, probs=probs)
        return tokens, probs


def random_weights(shape: Shape, seed: int, device) -> dict:
    g = torch.Generator().manual_seed(seed)
    s = shape

    def normal(*size, gain):
        return (torch.randn(*size, generator=g) * gain).to(torch.bfloat16).to(device)

    return dict(embed=normal(s.V, s.H, gain=1.0), qkv=normal(s.H, (s.Hq + 2 * s.Hkv) * s.D, gain=s.H ** -0.5),
                out=normal(s.Hq * s.D, s.H, gain=(s.Hq * s.D) ** -0.5), lm_head=normal(s.V, s.H, gain=3.0 * s.H ** -0.5),
                q_norm=torch.ones(s.D, device=device), k_norm=torch.ones(s.D, device=device))


def perturbed(weights: dict, amount: float, seed: int) -> dict:
    g = torch.Generator().manual_seed(seed)

    def moved(v):
        x = v.float().cpu()
        return (x + amount * x.std(correction=0) * torch.randn(v.shape, generator=g)).to(v)

    return {name: moved(v) for name, v in weights.items()}


def serve(shape: Shape, weights: dict, draft_weights: dict, prompts: list, sampling: Sampling, gamma: int, rounds: int,
          seed: int = 0, trace=None):
    """Serves the prompts (lists of token ids) for some rounds of speculation; returns each request's tokens.

    `trace`, if given, is called after each target pass with (requests' tokens, first positions of the window,
    window tokens [B, N] or None for the prompts, logits)."""
    dev = weights["embed"].device
    B, page = len(prompts), shape.page
    lens = [len(p) for p in prompts]
    pages = [-(-(n + (rounds + 1) * (gamma + 1)) // page) for n in lens]
    table = torch.zeros(B, max(pages), dtype=torch.int32)
    first = 0
    for b in range(B):
        table[b, :pages[b]] = torch.arange(first, first + pages[b], dtype=torch.int32)
        first += pages[b]
    target, draft = Model(shape, weights, first), Model(shape, draft_weights, first)
    block_table = table.to(dev)
    gen = torch.Generator().manual_seed(seed)
    uniforms = lambda n: torch.rand(n, generator=gen).to(dev)

    def places(positions):                                  # positions [B, N] -> slots [B, N]
        at = torch.gather(block_table, 1, (positions // page).long())
        return at * page + positions % page

    # prompts, packed
    tokens = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=dev)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32)
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])
    owner = torch.repeat_interleave(torch.arange(B), torch.tensor(lens))
    slots = (table[owner, (positions // page).long()] * page + positions % page).to(dev)
    positions = positions.to(dev)
    logits = target.prompt(tokens, positions, slots, cu.to(dev))
    draft.append(tokens, positions, slots)
    text = [list(p) for p in prompts]
    if trace:
        trace(text, [0] * B, None, logits)
    last, _ = sampling(logits[cu[1:].long().to(dev) - 1], uniforms(B))
    length = torch.tensor(lens, dtype=torch.int32, device=dev)
    for b, t in enumerate(last.tolist()):
        text[b].append(t)

    step = torch.arange(gamma + 1, dtype=torch.int32, device=dev)
    accepted_total = 0
    for r in range(rounds):
        # the draft: gamma tokens, one at a time
        window = torch.empty(B, gamma + 1, dtype=torch.int32, device=dev)
        p_draft = torch.empty(B, gamma, shape.V, device=dev)
        window[:, 0] = last
        positions = length[:, None] + step
        slots = places(positions)
        for i in range(gamma):
            out = draft.window(window[:, i:i + 1], positions[:, i:i + 1], slots[:, i:i + 1], block_table, length + i + 1)
            window[:, i + 1], p_draft[:, i] = sampling(out, uniforms(B))
        draft.append(*(t[:, gamma].contiguous() for t in (window, positions, slots)))
        # the target: the window at once, then the decision
        logits = target.window(window, positions, slots, block_table, length + gamma + 1)
        if trace:
            trace(text, length.tolist(), window, logits)
        _, p_target = sampling(logits, uniforms(B * (gamma + 1)))
        out, accepted = ds.dspark_verify(p_target.view(B, gamma + 1, shape.V), p_draft, window[:, 1:].contiguous(), None,
                                         seed=seed, offset=r)
        length = length + accepted + 1
        last = torch.gather(out, 1, accepted[:, None].long())[:, 0]
        for b, (n, row) in enumerate(zip(accepted.tolist(), out.tolist())):
            text[b] += row[:n + 1]
            accepted_total += n
    return text, accepted_total / (B * rounds)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--gamma", type=int, default=4)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    shape = Shape()
    weights = random_weights(shape, a.seed, dev)
    g = torch.Generator().manual_seed(a.seed + 1)
    prompts = [torch.randint(shape.V, (int(n),), generator=g).tolist() for n in torch.randint(1, 200, (a.requests,), generator=g)]
    full = lambda x, dtype=torch.float32: torch.full((a.requests,), x, dtype=dtype, device=dev)
    sampling = Sampling(full(0.8), full(50, torch.int32), full(0.95), full(0.0))
    text, accepted = serve(shape, weights, perturbed(weights, 0.02, a.seed + 2), prompts, sampling, a.gamma, a.rounds, a.seed)
    for p, t in zip(prompts, text):
        print(f"prompt of {len(p)} tokens -> {t[len(p):]}")
    print(f"{accepted:.2f} of {a.gamma} draft tokens accepted per round")


if __name__ == "__main__":
    main()
