"""Cases of the serving operators around the draft and verification path, with their plain forms.

Four operators: appending rotated keys and values to a paged cache, attention of a window of new
tokens over that cache, attention within packed prompts, and truncated sampling from logits.
`run` computes a case in elementary torch operations in 32 bits, or, where `own` is true, through
the framework's entry points; `exact` computes it in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MASS_BITS = 40            # a weight of 1 is 2^40 units of mass
FRAC_BITS = 24            # top-p and the uniform as integers over 2^24


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # one new token of one request: the smallest call of a decode loop, all latency
        dict(name="append_one", op="append", T=1, pad=0, Hq=32, Hkv=8, D=128, rot=128, page=16, slots=4096,
             dtype="bf16", interleaved=False, norm=False),
        # the verification batch of 64 requests with windows of 17, some of the rows padding (slot -1),
        # heads normalised before the rotation
        dict(name="append_verify", op="append", T=1088, pad=201, Hq=32, Hkv=8, D=128, rot=128, page=16, slots=16384,
             dtype="bf16", interleaved=False, norm=True),
        # a long prompt's tokens, half of each head rotated, pairs interleaved
        dict(name="append_prompt", op="append", T=8191, pad=0, Hq=32, Hkv=8, D=128, rot=64, page=64, slots=32768,
             dtype="f16", interleaved=True, norm=False),
        # decode of one request: one token over a few thousand cached ones, split over all SMs
        dict(name="decode_one", op="paged", B=1, N=1, Lmin=4097, Lmax=4097, Hq=32, Hkv=8, D=128, page=16, dtype="bf16",
             causal=True, ragged=False, mix=1),
        # the draft backbone's block of 8 tokens for many requests, every token seeing the whole block
        dict(name="draft_block", op="paged", B=200, N=8, Lmin=9, Lmax=2000, Hq=16, Hkv=4, D=64, page=32, dtype="f16",
             causal=False, ragged=False, mix=2),
        # verification windows of up to 17 tokens at the batched workload's 64 requests, ragged lengths
        dict(name="verify_window", op="paged", B=64, N=17, Lmin=100, Lmax=8000, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", causal=True, ragged=True, mix=3),
        # single-token decode over long contexts: the cache's bytes are all the time
        dict(name="decode_long", op="paged", B=5, N=1, Lmin=70000, Lmax=131071, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", causal=True, ragged=False, mix=4),
        # a few short prompts packed together: launch and tail costs
        dict(name="prompt_short", op="prompt", B=5, nmin=1, nmax=300, Hq=32, Hkv=8, D=128, dtype="bf16", causal=True, mix=5),
        # many prompts of different lengths, one key head per query head
        dict(name="prompt_packed", op="prompt", B=16, nmin=33, nmax=2048, Hq=16, Hkv=16, D=64, dtype="f16", causal=True,
             mix=6),
        # one long prompt: the tensor cores' rate
        dict(name="prompt_long", op="prompt", B=1, nmin=8192, nmax=8192, Hq=32, Hkv=8, D=128, dtype="bf16", causal=True,
             mix=7),
        # one row of the workloads' vocabulary: latency
        dict(name="sample_one", op="sample", R=1, V=151936, dtype="f32", probs=False),
        # the rows of the verification workload's shape at 64 requests, with the distributions that
        # verification takes
        dict(name="sample_verify", op="sample", R=576, V=151936, dtype="f32", probs=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "prompt", "prompt", "sample"])
    half = rng.choice(["bf16", "f16"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        T = _log_int(rng, 1, 8191)
        return dict(op=op, T=T, pad=rng.choice([0, T // 5]), Hq=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice([D, D // 2]),
                    page=page, slots=page * (-(-T // page) + rng.randint(1, 64)), dtype=half,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.5)
    if op == "paged":
        B = _log_int(rng, 1, 256)
        N = rng.choice([1, 1, rng.randint(2, 17)])
        most = min(131071, (5 * 70000 * 8 * 128) // (B * Hkv * D))
        Lmax = _log_int(rng, N + 1, most)
        return dict(op=op, B=B, N=N, Lmin=rng.choice([max(1, Lmax // 10), Lmax]), Lmax=Lmax, Hq=Hkv * G, Hkv=Hkv, D=D,
                    page=page, dtype=half, causal=rng.random() < 0.7, ragged=rng.random() < 0.5, mix=rng.randrange(1 << 20))
    if op == "prompt":
        G = min(G, max(1, 32 // Hkv))
        B = _log_int(rng, 1, 24)
        most = int(8192 / math.sqrt(B))
        nmax = _log_int(rng, 16, min(most, 8192))
        return dict(op=op, B=B, nmin=rng.choice([1, nmax]), nmax=nmax, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=half,
                    causal=rng.random() < 0.8, mix=rng.randrange(1 << 20))
    R = _log_int(rng, 1, 576)
    return dict(op=op, R=R, V=_log_int(rng, 1000, 151936), dtype=rng.choice(["f32", "bf16"]), probs=rng.random() < 0.5)


def _kv_lens(c):
    """Cached tokens of each request, the window's own among them."""
    rng = random.Random(c["mix"])
    lens = [_log_int(rng, c["Lmin"], c["Lmax"]) for _ in range(c["B"])]
    lens[0] = c["Lmax"]
    return lens


def _windows(c):
    """New tokens of each request: N of them, or where the scheduler admits fewer, 1 to N."""
    rng = random.Random(c["mix"] + 1)
    return [min(rng.randint(1, c["N"]) if c["ragged"] else c["N"], L) for L in _kv_lens(c)]


def _prompt_lens(c):
    rng = random.Random(c["mix"])
    lens = [_log_int(rng, c["nmin"], c["nmax"]) for _ in range(c["B"])]
    lens[0] = c["nmax"]
    return lens


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case)
    {"append": _prepare_append, "paged": _prepare_paged, "prompt": _prepare_prompt,
     "sample": _prepare_sample}[case["op"]](case, gen, state)
    return state


def _normal(gen, *shape, dtype=torch.float32, gain=1.0):
    x = torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=gen)
    return x.mul_(gain) if gain != 1.0 else x


def _projection(c, gen, T):
    """The fused projection's rows [T, (Hq + 2 Hkv) D] and the q, k, v views of it."""
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    rows = _normal(gen, T, (Hq + 2 * Hkv) * D, dtype=DTYPES[c["dtype"]])
    q, k, v = rows.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    return q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D)


def _prepare_append(c, gen, s):
    T, D, dt = c["T"], c["D"], DTYPES[c["dtype"]]
    s["q"], s["k"], s["v"] = _projection(c, gen, T)
    pages = c["slots"] // c["page"]
    s["k_cache"] = _normal(gen, pages, c["Hkv"], c["page"], D, dtype=dt)
    s["v_cache"] = _normal(gen, pages, c["Hkv"], c["page"], D, dtype=dt)
    slots = torch.randperm(pages * c["page"], generator=gen, device="cuda")[:T]
    at = torch.randperm(T, generator=gen, device="cuda")[:c["pad"]]
    s["slots"] = slots.index_fill(0, at, -1).to(torch.int32)
    positions = 16384
    s["positions"] = torch.randint(0, positions, (T,), generator=gen, device="cuda", dtype=torch.int32)
    freq = 1e6 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    s["q_norm"] = _normal(gen, D).mul_(0.1).add_(1.0) if c["norm"] else None
    s["k_norm"] = _normal(gen, D).mul_(0.1).add_(1.0) if c["norm"] else None


def _prepare_paged(c, gen, s):
    B, N, D, page, dt = c["B"], c["N"], c["D"], c["page"], DTYPES[c["dtype"]]
    lens, windows = _kv_lens(c), _windows(c)
    need = [-(-n // page) for n in lens]
    width, total = max(need), sum(need)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    s["block_table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["lengths"] = torch.tensor(windows, dtype=torch.int32, device="cuda") if c["ragged"] or min(windows) < N else None
    s["q"] = _normal(gen, B, N, c["Hq"], D, dtype=dt, gain=2.0)
    s["k_cache"] = _normal(gen, total, c["Hkv"], page, D, dtype=dt)
    s["v_cache"] = _normal(gen, total, c["Hkv"], page, D, dtype=dt)
    # the slots behind a request's last token were never written
    last = torch.tensor([row[n - 1] for row, n in zip(table, need)], device="cuda")
    rest = torch.tensor([L - (n - 1) * page for L, n in zip(lens, need)], device="cuda")
    stale = torch.arange(page, device="cuda")[None, None, :, None] >= rest[:, None, None, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[last] = torch.where(stale, torch.full_like(cache[:1], math.nan), cache[last])
    s["scale"] = D ** -0.5


def _prepare_prompt(c, gen, s):
    lens = _prompt_lens(c)
    s["q"], s["k"], s["v"] = _projection(c, gen, sum(lens))
    s["q"].mul_(2.0)
    s["cu_seqlens"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    s["scale"] = c["D"] ** -0.5


def _prepare_sample(c, gen, s):
    R, V = c["R"], c["V"]
    s["logits"] = _normal(gen, R, V, gain=3.0).to(DTYPES[c["dtype"]])

    def pick(values, dtype):
        at = torch.randint(0, len(values), (R,), generator=gen, device="cuda")
        return torch.tensor(values, dtype=dtype, device="cuda")[at]

    # the settings that requests bring: some greedy, some with one filter, some with all
    s["temperature"] = pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2], torch.float32)
    s["top_k"] = pick([0, 0, 20, 50, 1000], torch.int32)
    s["top_p"] = pick([1.0, 0.95, 0.9, 0.8], torch.float32)
    s["min_p"] = pick([0.0, 0.0, 0.0, 0.05], torch.float32)
    s["u"] = torch.rand(R, generator=gen, device="cuda")


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        return {"append": _own_append, "paged": _own_paged, "prompt": _own_prompt, "sample": _own_sample}[op](state)
    return {"append": _plain_append, "paged": _plain_paged, "prompt": _plain_prompt, "sample": _plain_sample}[op](state)


def _own_append(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    if "workspace" not in s:
        s["workspace"] = ds.Workspace(ds.OP_KV_APPEND)
    q = ds.dspark_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["k_cache"], s["v_cache"],
                            interleaved=s["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                            workspace=s["workspace"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_paged(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    if "workspace" not in s:
        s["workspace"] = ds.Workspace(ds.OP_PAGED_ATTENTION, s["B"], s["N"], s["Hq"], s["D"])
    lse = torch.empty(s["B"], s["N"], s["Hq"], device="cuda")
    out = ds.dspark_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"], s["scale"],
                                    lengths=s["lengths"], causal=s["causal"], lse=lse, workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_prompt(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    if "workspace" not in s:
        s["workspace"] = ds.Workspace(ds.OP_PROMPT_ATTENTION, s["B"], s["q"].shape[0], s["Hq"], s["D"])
    lse = torch.empty(s["q"].shape[0], s["Hq"], device="cuda")
    out = ds.dspark_prompt_attention(s["q"], s["k"], s["v"], s["cu_seqlens"], s["scale"], causal=s["causal"], lse=lse,
                                     workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_sample(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    if "workspace" not in s:
        s["workspace"] = ds.Workspace(ds.OP_SAMPLE, s["R"], 1, s["V"])
    probs = torch.empty(s["R"], s["V"], device="cuda") if s["probs"] else None
    tokens = ds.dspark_sample(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], probs=probs,
                              workspace=s["workspace"])
    return {"tokens": tokens, "probs": probs} if s["probs"] else {"tokens": tokens}


# --------------------------------------------------------------------------------------------
# Plain forms, in 32 bits
# --------------------------------------------------------------------------------------------
def _rotate(x, cos_sin, interleaved):
    """The first `rot` values of each head turned by the token's angles; x [T, H, D]."""
    half = cos_sin.shape[1] // 2
    c, t = cos_sin[:, None, :half], cos_sin[:, None, half:]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    a, b = a * c - b * t, b * c + a * t
    turned = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _rms(x, weight, eps=1e-6):
    return x if weight is None else x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps) * weight


def _plain_append(s):
    cs = s["cos_sin"][s["positions"].long()]
    q = _rotate(_rms(s["q"].float(), s["q_norm"]), cs, s["interleaved"]).to(s["q"].dtype)
    k = _rotate(_rms(s["k"].float(), s["k_norm"]), cs, s["interleaved"]).to(s["k"].dtype)
    at = s["slots"].long()
    kept = at >= 0
    at, page = at[kept], s["page"]
    s["k_cache"][at // page, :, at % page] = k[kept]
    s["v_cache"][at // page, :, at % page] = s["v"][kept]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _softmax_rows(scores, seen):
    """Weights, their sum and the row's largest score where `seen`; rows that see nothing have sum 0."""
    scores = torch.where(seen, scores, -math.inf)
    m = scores.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(scores - m)
    return w, w.sum(dim=-1, keepdim=True), m


def _plain_paged(s):
    B, N, Hq, D = s["q"].shape
    Hkv, G = s["Hkv"], Hq // s["Hkv"]
    pages = s["block_table"].long().clamp(min=0)
    K = s["k_cache"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    V = s["v_cache"][pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D).float()
    j = torch.arange(K.shape[2], device="cuda")
    i = torch.arange(N, device="cuda")
    kv = s["kv_len"].long()[:, None]
    n = s["lengths"].long()[:, None] if s["lengths"] is not None else torch.full_like(kv, N)
    limit = kv - n + i + 1 if s["causal"] else kv.expand(B, N)
    limit = torch.where(i < n, limit, 0)                                       # [B, N]
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    scores = q @ K.transpose(-1, -2) * s["scale"]
    seen = (j < limit[..., None])[:, None, :, None, :].expand(B, 1, N, G, -1).reshape(B, 1, N * G, -1)
    w, total, m = _softmax_rows(scores, seen)
    V = torch.where((j < kv)[:, None, :, None], V, 0.0)
    out = torch.where(total > 0, w @ V / total, 0.0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)

    def rows(x):
        return x.view(B, Hkv, N, G, -1).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, -1)

    return {"out": rows(out).to(s["q"].dtype).contiguous(), "lse": rows(lse)[..., 0].contiguous()}


def _plain_prompt(s):
    T, Hq, D = s["q"].shape
    Hkv, G = s["Hkv"], Hq // s["Hkv"]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["cu_seqlens"].long(), t, right=True)
    seen = seq[:, None] == seq[None, :]
    if s["causal"]:
        seen = seen & (t[None, :] <= t[:, None])
    q = s["q"].float().view(T, Hkv, G, D).permute(1, 2, 0, 3)
    K = s["k"].float().permute(1, 2, 0)[:, None]
    V = s["v"].float().permute(1, 0, 2)[:, None]
    w, total, m = _softmax_rows(q @ K * s["scale"], seen)
    out = (w @ V / total).permute(2, 0, 1, 3).reshape(T, Hq, D).to(s["q"].dtype)
    lse = (m + torch.log(total))[..., 0].permute(2, 0, 1).reshape(T, Hq)
    return {"out": out.contiguous(), "lse": lse.contiguous()}


def _share(total, frac):
    """floor(total * frac / 2^FRAC_BITS) for total < 2^62 and frac in [0, 2^FRAC_BITS]."""
    low = (1 << FRAC_BITS) - 1
    return (total >> FRAC_BITS) * frac + (((total & low) * frac) >> FRAC_BITS)


def _plain_sample(s):
    x, order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    V = x.shape[1]
    rank = torch.arange(V, device="cuda")
    T = s["temperature"][:, None]
    greedy = T == 0
    w = torch.exp((x - x[:, :1]) * (1.0 / torch.where(greedy, 1.0, T)))
    mass = torch.floor(w * 2.0 ** MASS_BITS).long()
    k = s["top_k"].long()[:, None]
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))
    keep = (rank < k) & (w >= s["min_p"][:, None])
    mass = torch.where(keep, mass, 0)
    before = mass.cumsum(dim=1) - mass
    need = _share(mass.sum(dim=1, keepdim=True), torch.floor(s["top_p"][:, None] * 2.0 ** FRAC_BITS).long())
    mass = torch.where((before < need) | (rank == 0), mass, 0)
    total = mass.sum(dim=1, keepdim=True)
    target = _share(total, torch.floor(s["u"][:, None] * 2.0 ** FRAC_BITS).long())
    by_id = torch.zeros_like(mass).scatter_(1, order, mass)
    tokens = (by_id.cumsum(dim=1) <= target).sum(dim=1).to(torch.int32)
    if not s["probs"]:
        return {"tokens": tokens}
    w = torch.where(mass > 0, w, 0.0) / (total.float() * 2.0 ** -MASS_BITS)
    return {"tokens": tokens, "probs": torch.zeros_like(w).scatter_(1, order, w)}


# --------------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------------
def work(case):
    c, e = case, 4 if case["dtype"] == "f32" else 2
    if c["op"] == "append":
        written = c["T"] - c["pad"]
        per = (c["Hq"] + 2 * c["Hkv"]) * c["D"] * e
        bytes_ = c["T"] * per + (c["T"] * c["Hq"] + 2 * written * c["Hkv"]) * c["D"] * e + c["T"] * (8 + 4 * c["rot"])
        return {"bytes": bytes_, "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "paged":
        lens, windows = _kv_lens(c), _windows(c)
        rows = sum(windows)
        seen = sum(n * L - (n * (n - 1) // 2 if c["causal"] else 0) for n, L in zip(windows, lens))
        bytes_ = 2 * sum(lens) * c["Hkv"] * c["D"] * e + 2 * rows * c["Hq"] * c["D"] * e + 4 * rows * c["Hq"]
        return {"bytes": bytes_, "flops": 4 * c["D"] * c["Hq"] * seen}
    if c["op"] == "prompt":
        lens = _prompt_lens(c)
        seen = sum(n * (n + 1) // 2 if c["causal"] else n * n for n in lens)
        bytes_ = sum(lens) * ((2 * c["Hq"] + 2 * c["Hkv"]) * c["D"] * e + 4 * c["Hq"])
        return {"bytes": bytes_, "flops": 4 * c["D"] * c["Hq"] * seen}
    n = c["R"] * c["V"]
    return {"bytes": n * (e + (4 if c["probs"] else 0)), "flops": 4 * n}


# --------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# --------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "sample" and not case["probs"]:
        return None                                                            # whole numbers only
    s = prepare(case, seed)
    return {"append": _exact_append, "paged": _exact_paged, "prompt": _exact_prompt, "sample": _exact_sample}[case["op"]](s)


def _exact_append(s):
    angle = s["cos_sin"].double()[s["positions"].long()]
    half = angle.shape[1] // 2
    turn = torch.complex(angle[:, None, :half], angle[:, None, half:])

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()
        if s["interleaved"]:
            z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:-1], half, 2).contiguous()) * turn
            return torch.cat([torch.view_as_real(z).reshape(*x.shape[:-1], 2 * half), x[..., 2 * half:]], -1)
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
        return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)

    caches = []
    for cache, new in ((s["k_cache"], turned(s["k"], s["k_norm"])), (s["v_cache"], s["v"].double())):
        P, H, page, D = cache.shape
        flat = cache.double().transpose(1, 2).reshape(P * page, H, D)
        at = s["slots"].long()
        flat[at[at >= 0]] = new[at >= 0]
        caches.append(flat.view(P, page, H, D).transpose(1, 2).contiguous())
    return {"q": turned(s["q"], s["q_norm"]), "k_cache": caches[0], "v_cache": caches[1]}


def _exact_paged(s):
    B, N, Hq, D = s["q"].shape
    G = Hq // s["Hkv"]
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(_kv_lens(s), _windows(s))):
        pages = s["block_table"][b, :-(-L // s["page"])].long()
        for h in range(s["Hkv"]):
            k = s["k_cache"][pages, h].reshape(-1, D)[:L].double()
            v = s["v_cache"][pages, h].reshape(-1, D)[:L].double()
            q = s["q"][b, :n, h * G:(h + 1) * G].double()
            z = torch.einsum("igd,jd->gij", q, k) * s["scale"]
            if s["causal"]:
                hidden = torch.arange(L, device="cuda")[None] > torch.arange(L - n, L, device="cuda")[:, None]
                z = z.masked_fill(hidden, -math.inf)
            total = torch.logsumexp(z, dim=-1, keepdim=True)
            out[b, :n, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", (z - total).exp(), v)
            lse[b, :n, h * G:(h + 1) * G] = total[..., 0].T
    return {"out": out, "lse": lse}


def _exact_prompt(s):
    T, Hq, D = s["q"].shape
    G = Hq // s["Hkv"]
    out = torch.empty(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, Hq, dtype=torch.float64, device="cuda")
    at = 0
    for n in _prompt_lens(s):
        rows = slice(at, at + n)
        hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1) if s["causal"] else None
        for h in range(Hq):
            z = s["q"][rows, h].double() @ s["k"][rows, h // G].double().T * s["scale"]
            if hidden is not None:
                z = z.masked_fill_(hidden, -math.inf)
            total = torch.logsumexp(z, dim=-1, keepdim=True)
            out[rows, h] = z.sub_(total).exp_() @ s["v"][rows, h // G].double()
            lse[rows, h] = total[:, 0]
        at += n
    return {"out": out, "lse": lse}


def _exact_sample(s):
    probs = torch.zeros(s["R"], s["V"], dtype=torch.float64, device="cuda")
    for r in range(s["R"]):
        x = s["logits"][r].double()
        T, k, p, least = (float(s[name][r]) for name in ("temperature", "top_k", "top_p", "min_p"))
        x, order = torch.sort(x, descending=True, stable=True)
        if T == 0.0:
            probs[r, order[0]] = 1.0
            continue
        w = ((x - x[0]) / T).exp()
        if k > 0:
            w = w[:int(k)]
        w = w[w >= least]
        before = (w.cumsum(0) - w) / w.sum()
        w = w[(before < p) | (before == 0)]
        probs[r, order[:w.numel()]] = w / w.sum()
    return {"tokens": None, "probs": probs}
