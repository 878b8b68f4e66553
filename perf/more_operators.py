"""Cases of the operators that draft and verify trees of tokens, with their plain forms.

Five operators: attention of a tree of drafted tokens over a paged cache, attention with a sliding
window and sinks over it, verification of a tree, moving the accepted path's keys and values
together, and copying pages for sequences that part.  `run` computes a case in elementary torch
operations in 32 bits, or, where `own` is true, through the framework's entry points; `exact`
computes it in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MASS_BITS = 40            # a weight of 1 is 2^40 units of mass
FRAC_BITS = 24            # the uniform as an integer over 2^24
DEPTH = 8                 # of the drafted trees, the root not counted


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # the drafted tree of one request over a short context: the smallest verification pass, all latency
        dict(name="tree_one", op="attend", tree=True, B=1, N=25, Lmin=1051, Lmax=1051, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", window=0, sinks=0, causal=True, ragged=False, mix=1),
        # trees of up to 64 nodes for a batch of requests: two tiles of rows per key head
        dict(name="tree_batch", op="attend", tree=True, B=16, N=64, Lmin=500, Lmax=8000, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", window=0, sinks=0, causal=True, ragged=True, mix=2),
        # a layer with a window in the same serving loop, trees over long contexts
        dict(name="tree_window", op="attend", tree=True, B=33, N=31, Lmin=2000, Lmax=32000, Hq=16, Hkv=4, D=64, page=32,
             dtype="f16", window=2048, sinks=4, causal=True, ragged=True, mix=3),
        # single-token decode of long contexts that sees a window and four sinks
        dict(name="window_decode", op="attend", tree=False, B=64, N=1, Lmin=4001, Lmax=65536, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", window=1024, sinks=4, causal=True, ragged=False, mix=4),
        # a chunk of a long prompt, appended to its cache and then attended with a window: the tensor cores' rate
        dict(name="window_chunk", op="attend", tree=False, B=2, N=4096, Lmin=9999, Lmax=20000, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", window=1024, sinks=16, causal=True, ragged=False, mix=5),
        # one tree of one request, greedy: a chain of rows, all latency
        dict(name="verify_one", op="verify", B=1, N=25, V=151936, dtype="f32", greedy=True, tokens=False, ragged=False, mix=6),
        # the batched workload's 64 requests, each with its own temperature
        dict(name="verify_batch", op="verify", B=64, N=64, V=151936, dtype="f32", greedy=False, tokens=False, ragged=True,
             mix=7),
        # the target's tokens were sampled with top-p and top-k before: only the walk is left
        dict(name="verify_tokens", op="verify", B=64, N=64, V=151936, dtype="f32", greedy=False, tokens=True, ragged=True,
             mix=8),
        # the accepted path of one request in one layer's cache
        dict(name="compact_one", op="compact", B=1, N=25, layers=1, Lmin=1051, Lmax=1051, Hkv=8, D=128, page=16,
             dtype="bf16", ragged=False, mix=9),
        # the accepted paths of a batch in all layers at once
        dict(name="compact_batch", op="compact", B=64, N=64, layers=24, Lmin=64, Lmax=300, Hkv=8, D=128, page=16,
             dtype="bf16", ragged=True, mix=10),
        # a sequence parts in two: its last page, partly filled, is copied in one layer's cache
        dict(name="copy_one", op="copy", M=1, pages=64, layers=1, Hkv=8, D=128, page=16, dtype="bf16", partial=True, mix=11),
        # many sequences part, or are moved to other pages, in all layers
        dict(name="copy_many", op="copy", M=500, pages=1200, layers=24, Hkv=8, D=128, page=16, dtype="bf16", partial=False,
             mix=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "window", "window", "verify", "compact", "copy"])
    half = rng.choice(["bf16", "f16"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    if op == "tree":
        B = _log_int(rng, 1, 64)
        N = _log_int(rng, 1, 128)
        Lmax = _log_int(rng, N + 1, min(32000, 16 * 8000 * 64 * 32 * 128 // (B * N * Hkv * G * D)) + N + 1)
        return dict(op="attend", tree=True, B=B, N=N, Lmin=max(N, Lmax // rng.choice([1, 10])), Lmax=Lmax, Hq=Hkv * G, Hkv=Hkv,
                    D=D, page=page, dtype=half, window=rng.choice([0, 0, N + _log_int(rng, 1, 2048)]), sinks=rng.choice([0, 4, 130]),
                    causal=True, ragged=rng.random() < 0.6, mix=mix)
    if op == "window":
        B = _log_int(rng, 1, 64)
        N = rng.choice([1, rng.randint(2, 17), _log_int(rng, 18, max(19, 8000 // B))])
        Lmax = N + _log_int(rng, 1, max(2, min(65536, 4000000 // B)))
        return dict(op="attend", tree=False, B=B, N=N, Lmin=max(1, Lmax // rng.choice([1, 10])), Lmax=Lmax, Hq=min(32, Hkv * G) // Hkv * Hkv,
                    Hkv=Hkv, D=D, page=page, dtype=half, window=_log_int(rng, 1, 1024), sinks=rng.choice([0, 4, 16, 130]),
                    causal=rng.random() < 0.8, ragged=rng.random() < 0.4, mix=mix)
    if op == "verify":
        return dict(op=op, B=_log_int(rng, 1, 64), N=_log_int(rng, 1, 64), V=_log_int(rng, 1000, 151936),
                    dtype=rng.choice(["f32", "bf16"]), greedy=rng.random() < 0.3, tokens=rng.random() < 0.3,
                    ragged=rng.random() < 0.5, mix=mix)
    layers = rng.randint(1, 24)
    if op == "compact":
        N = _log_int(rng, 1, 64)
        return dict(op=op, B=_log_int(rng, 1, 64), N=N, layers=layers, Lmin=N, Lmax=N + rng.randint(0, 236), Hkv=Hkv, D=D,
                    page=page, dtype=half, ragged=rng.random() < 0.5, mix=mix)
    most = 1200 * 16 // page
    pages = _log_int(rng, 2, most)
    return dict(op=op, M=_log_int(rng, 1, pages // 2), pages=pages, layers=layers, Hkv=Hkv, D=D, page=page, dtype=half,
                partial=rng.random() < 0.5, mix=mix)


def _kv_lens(c):
    """Cached tokens of each request, the window's own among them."""
    rng = random.Random(c["mix"])
    lens = [_log_int(rng, c["Lmin"], c["Lmax"]) for _ in range(c["B"])]
    lens[0] = c["Lmax"]
    return lens


def _windows(c):
    """New tokens of each request: N of them, or where requests bring fewer, 0 (rarely) to N."""
    rng = random.Random(c["mix"] + 1)
    lens = _kv_lens(c) if "Lmin" in c else [c["N"]] * c["B"]
    own_n = [max(0, rng.randint(-c["N"] // 16, c["N"])) if c["ragged"] else c["N"] for _ in lens]
    own_n[0] = c["N"]
    return [min(n, L) for n, L in zip(own_n, lens)]


def _trees(c):
    """Parent and depth of every node: node 0 is the root, later ones hang from any that is not too deep."""
    rng = random.Random(c["mix"] + 2)
    parents, depths = [], []
    for _ in range(c["B"]):
        parent, depth = [-1], [0]
        for i in range(1, c["N"]):
            p = rng.randrange(i)
            while depth[p] >= DEPTH:
                p = rng.randrange(i)
            parent.append(p)
            depth.append(depth[p] + 1)
        parents.append(parent)
        depths.append(depth)
    return parents, depths


def _paths(c):
    """The accepted path of each request: the root's way to one of its nodes (empty without nodes)."""
    rng = random.Random(c["mix"] + 3)
    parents, _ = _trees(c)
    paths = []
    for b, n in enumerate(_windows(c)):
        at = rng.randrange(n) if n else -1
        path = []
        while at >= 0:
            path.append(at)
            at = parents[b][at]
        paths.append(path[::-1])
    return paths


def _used(c):
    """Tokens of each copied page that are filled."""
    rng = random.Random(c["mix"])
    return [rng.randint(0 if c["M"] > 1 else 1, c["page"]) if c["partial"] else c["page"] for _ in range(c["M"])]


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case)
    {"attend": _prepare_attend, "verify": _prepare_verify, "compact": _prepare_compact, "copy": _prepare_copy}[case["op"]](
        case, gen, state)
    return state


def _normal(gen, *shape, dtype=torch.float32, gain=1.0):
    x = torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=gen)
    return x.mul_(gain) if gain != 1.0 else x


def _ints(rows):
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def _table(c, gen, lens):
    """A block table of pages in random order, and how many pages it names."""
    need = [-(-n // c["page"]) for n in lens]
    width, total = max(max(need), 1), max(sum(need), 1)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return table, need, total


def _prepare_attend(c, gen, s):
    B, N, D, page, dt = c["B"], c["N"], c["D"], c["page"], DTYPES[c["dtype"]]
    lens, windows = _kv_lens(c), _windows(c)
    table, need, total = _table(c, gen, lens)
    s["block_table"], s["kv_len"] = _ints(table), _ints(lens)
    s["lengths"] = _ints(windows) if c["ragged"] or min(windows) < N else None
    if c["tree"]:
        s["parents"] = _ints(_trees(c)[0])
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


def _prepare_verify(c, gen, s):
    B, N, V = c["B"], c["N"], c["V"]
    s["parents"] = _ints(_trees(c)[0])
    s["lengths"] = _ints(_windows(c)) if c["ragged"] else None
    s["draft_tokens"] = torch.randint(0, V, (B, N), generator=gen, device="cuda", dtype=torch.int32)
    # along the accepted path the target is nearly sure of the drafted token
    at = [(b, p, x) for b, path in enumerate(_paths(c)) for p, x in zip(path, path[1:])]
    rows = torch.tensor([[b, p, b, x] for b, p, x in at], dtype=torch.long, device="cuda").view(-1, 4).T
    if c["tokens"]:
        s["target_tokens"] = torch.randint(0, V, (B, N), generator=gen, device="cuda", dtype=torch.int32)
        s["target_tokens"][rows[0], rows[1]] = s["draft_tokens"][rows[2], rows[3]]
        return
    s["target"] = _normal(gen, B, N, V, dtype=DTYPES[c["dtype"]], gain=3.0)
    s["target"][rows[0], rows[1], s["draft_tokens"][rows[2], rows[3]].long()] = 30.0
    s["temperature"] = s["u"] = None
    if not c["greedy"]:
        kinds = torch.tensor([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2], device="cuda")
        s["temperature"] = kinds[torch.randint(0, len(kinds), (B,), generator=gen, device="cuda")]
        s["u"] = torch.rand(B, N, generator=gen, device="cuda")


def _prepare_compact(c, gen, s):
    dt, lens, N = DTYPES[c["dtype"]], _kv_lens(c), c["N"]
    table, _, total = _table(c, gen, lens)
    s["block_table"], s["kv_len"] = _ints(table), _ints(lens)
    s["lengths"] = _ints(_windows(c)) if c["ragged"] else None
    paths = _paths(c)
    s["path"] = _ints([p + [-1] * (N - len(p)) for p in paths])
    s["num_accepted"] = _ints([max(0, len(p) - 1) for p in paths])
    s["k_cache"] = _normal(gen, c["layers"], total, c["Hkv"], c["page"], c["D"], dtype=dt)
    s["v_cache"] = _normal(gen, c["layers"], total, c["Hkv"], c["page"], c["D"], dtype=dt)


def _prepare_copy(c, gen, s):
    dt = DTYPES[c["dtype"]]
    s["k_cache"] = _normal(gen, c["layers"], c["pages"], c["Hkv"], c["page"], c["D"], dtype=dt)
    s["v_cache"] = _normal(gen, c["layers"], c["pages"], c["Hkv"], c["page"], c["D"], dtype=dt)
    order = torch.randperm(c["pages"], generator=gen, device="cuda").to(torch.int32)
    # some sources are copied more than once, as a sequence that parts in several does
    among = torch.randint(0, c["pages"] - c["M"], (c["M"],), generator=gen, device="cuda")
    s["dst"], s["src"] = order[:c["M"]].contiguous(), order[c["M"]:][among].contiguous()
    s["used"] = _ints(_used(c)) if c["partial"] else None


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        return {"attend": _own_attend, "verify": _own_verify, "compact": _own_compact, "copy": _own_copy}[op](state)
    return {"attend": _plain_attend, "verify": _plain_verify, "compact": _plain_compact, "copy": _plain_copy}[op](state)


def _own_attend(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    lse = torch.empty(s["B"], s["N"], s["Hq"], device="cuda")
    if s["tree"]:
        if "workspace" not in s:
            s["workspace"] = ds.Workspace(ds.OP_TREE_ATTENTION, s["B"], s["N"], s["Hq"], s["D"])
        out = ds.dspark_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"], s["parents"],
                                       s["scale"], lengths=s["lengths"], window=s["window"], sinks=s["sinks"], lse=lse,
                                       workspace=s["workspace"])
    else:
        if "workspace" not in s:
            s["workspace"] = ds.Workspace(ds.OP_WINDOW_ATTENTION, s["B"], s["N"], s["Hq"], s["D"])
        out = ds.dspark_window_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"], s["window"],
                                         s["sinks"], s["scale"], lengths=s["lengths"], causal=s["causal"], lse=lse,
                                         workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_verify(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    if "workspace" not in s:
        s["workspace"] = ds.Workspace(ds.OP_VERIFY_TREE, s["B"], s["N"])
    if s["tokens"]:
        out = ds.dspark_verify_tree_tokens(s["target_tokens"], s["parents"], s["draft_tokens"], lengths=s["lengths"],
                                           workspace=s["workspace"])
    else:
        out = ds.dspark_verify_tree(s["target"], s["parents"], s["draft_tokens"], temperature=s["temperature"], u=s["u"],
                                    lengths=s["lengths"], workspace=s["workspace"])
    return dict(zip(("out_tokens", "num_accepted", "path"), out))


def _own_compact(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    if "workspace" not in s:
        s["workspace"] = ds.Workspace(ds.OP_KV_COMPACT)
    kv_len = ds.dspark_kv_compact(s["k_cache"], s["v_cache"], s["block_table"], s["kv_len"], s["path"], s["num_accepted"],
                                  lengths=s["lengths"], workspace=s["workspace"])
    return {"kv_len": kv_len, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_copy(s):
    import draft_sampling_verification_tcgen05_gb300 as ds
    if "workspace" not in s:
        s["workspace"] = ds.Workspace(ds.OP_KV_COPY_PAGES)
    ds.dspark_kv_copy_pages(s["k_cache"], s["v_cache"], s["src"], s["dst"], used=s["used"], workspace=s["workspace"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# --------------------------------------------------------------------------------------------
# Plain forms, in 32 bits
# --------------------------------------------------------------------------------------------
def _lengths(s):
    return s["lengths"].long() if s["lengths"] is not None else torch.full((s["B"],), s["N"], device="cuda")


def _ancestors(parents):
    """[B, N, N] truth values (m is i or an ancestor of i), and the nodes' depths."""
    B, N = parents.shape
    at = torch.arange(N, device="cuda").expand(B, N)
    sees = torch.zeros(B, N, N + 1, dtype=torch.bool, device="cuda")
    for _ in range(min(N, DEPTH + 1)):
        sees.scatter_(2, at[..., None], True)
        at = torch.where(at == N, N, parents.long().gather(1, at.clamp(max=N - 1)))
        at = torch.where(at < 0, N, at)
    sees = sees[..., :N]
    return sees, sees.sum(dim=2) - 1


def _plain_attend(s):
    B, N, Hq, D = s["q"].shape
    Hkv, G = s["Hkv"], Hq // s["Hkv"]
    kv, n = s["kv_len"].long()[:, None], _lengths(s)[:, None]
    base = kv - n
    i = torch.arange(N, device="cuda")
    if s["tree"]:
        sees, depth = _ancestors(s["parents"])
    else:
        sees = (i[None, :] <= i[:, None]) if s["causal"] else torch.ones(N, N, dtype=torch.bool, device="cuda")
        sees, depth = sees.expand(B, N, N), i.expand(B, N)
    # the tokens that any row of a request can see: with a window the sinks and the last of them
    W, sinks = s["window"], s["sinks"]
    if W:
        behind = base - W + 1 + torch.arange(W - 1 + N, device="cuda")
        j = torch.cat([torch.arange(sinks, device="cuda").expand(B, sinks), behind], dim=1)
        there = torch.cat([(j < kv)[:, :sinks], ((behind >= sinks) & (behind < kv))], dim=1)
    else:
        j = torch.arange(s["block_table"].shape[1] * s["page"], device="cuda").expand(B, -1)
        there = j < kv
    j = j.clamp(0, s["block_table"].shape[1] * s["page"] - 1)
    pages = s["block_table"].long().gather(1, j // s["page"]).clamp(min=0)
    K = s["k_cache"][pages, :, j % s["page"]].float().transpose(1, 2)                       # [B, Hkv, S, D]
    V = s["v_cache"][pages, :, j % s["page"]].float().transpose(1, 2)
    m = j - base                                                                            # place among the new tokens
    seen = sees.gather(2, m.clamp(0, N - 1)[:, None].expand(B, N, -1)) | (m < 0)[:, None]
    if W:
        seen = seen & ((j < sinks)[:, None] | (j[:, None] > (base + depth)[..., None] - W))
    seen = seen & there[:, None] & (i[None, :, None] < n[..., None])
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    scores = (q @ K.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, N, G, -1)
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = scores.sub_(top).exp_()
    total = w.sum(dim=-1, keepdim=True)
    V = torch.where(there[:, None, :, None], V, 0.0)
    out = (w.view(B, Hkv, N * G, -1) @ V).view(B, Hkv, N, G, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype).contiguous(),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, N, Hq).contiguous()}


def _share(total, frac):
    """floor(total * frac / 2^FRAC_BITS) for total < 2^62 and frac in [0, 2^FRAC_BITS]."""
    low = (1 << FRAC_BITS) - 1
    return (total >> FRAC_BITS) * frac + (((total & low) * frac) >> FRAC_BITS)


def _target_token(s, node):
    """The target's token behind `node` of every request."""
    if s["tokens"]:
        return s["target_tokens"].long().gather(1, node[:, None])[:, 0]
    x = s["target"][torch.arange(s["B"], device="cuda"), node].float()
    first = x.argmax(dim=1)
    if s["temperature"] is None:
        return first
    T = s["temperature"][:, None]
    w = torch.exp((x - x.amax(dim=1, keepdim=True)) * (1.0 / torch.where(T == 0, 1.0, T)))
    mass = torch.floor(w * 2.0 ** MASS_BITS).long()
    u = torch.floor(s["u"].gather(1, node[:, None]) * 2.0 ** FRAC_BITS).long()
    target = _share(mass.sum(dim=1, keepdim=True), u)
    return torch.where(T[:, 0] == 0, first, (mass.cumsum(dim=1) <= target).sum(dim=1))


def _plain_verify(s):
    B, N = s["draft_tokens"].shape
    n = _lengths(s)
    node = torch.zeros(B, dtype=torch.long, device="cuda")
    walking = n > 0
    tokens = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    accepted = torch.zeros(B, dtype=torch.int32, device="cuda")
    i = torch.arange(N, device="cuda")
    for k in range(min(N, DEPTH + 1)):
        y = _target_token(s, node)
        tokens[:, k] = torch.where(walking, y, -1).int()
        path[:, k] = torch.where(walking, node, -1).int()
        child = (s["parents"] == node[:, None]) & (s["draft_tokens"] == y[:, None]) & (i < n[:, None])
        walking = walking & child.any(dim=1)
        accepted += walking.int()
        node = torch.where(walking, child.int().argmax(dim=1), node)
    return {"out_tokens": tokens, "num_accepted": accepted, "path": path}


def _plain_compact(s):
    base = (s["kv_len"].long() - _lengths(s))[:, None]
    i = torch.arange(s["N"], device="cuda")
    moved = (i >= 1) & (i <= s["num_accepted"].long()[:, None])
    page = s["page"]

    def place(at):
        at = at[moved]
        b = torch.arange(s["B"], device="cuda")[:, None].expand(moved.shape)[moved]
        return s["block_table"].long()[b, at // page], at % page

    src, dst = place(base + s["path"].long()), place(base + i)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, dst[0], :, dst[1]] = cache[:, src[0], :, src[1]]
    kept = torch.where(_lengths(s) > 0, base[:, 0] + 1 + s["num_accepted"], base[:, 0])
    return {"kv_len": kept.int(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for cache in (s["k_cache"], s["v_cache"]):
        new = cache[:, src]
        if s["used"] is not None:
            filled = torch.arange(s["page"], device="cuda")[:, None] < s["used"].long()[:, None, None, None]
            new = torch.where(filled, new, cache[:, dst])
        cache[:, dst] = new
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# --------------------------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------------------------
def work(case):
    c, e = case, 4 if case["dtype"] == "f32" else 2
    if c["op"] == "attend":
        lens, windows = _kv_lens(c), _windows(c)
        _, depths = _trees(c) if c["tree"] else (None, [range(c["N"])] * c["B"])
        W, sinks = c["window"], c["sinks"]
        read = seen = 0
        for L, n, depth in zip(lens, windows, depths):
            if n == 0:
                continue
            base, far = L - n, max(depth[:n])
            rows = [base + depth[i] for i in range(n)]                       # position of each row
            own = [n if not c["causal"] else depth[i] + 1 for i in range(n)] # what it sees of the new tokens
            if not W:
                read += L
                seen += sum(base + o for o in own)
                continue
            low = max(sinks, base - W + 1)                                   # the first row's oldest token
            read += min(sinks, L) + max(0, L - low)
            for p, o in zip(rows, own):
                old = p - W + 1                                              # its oldest one in the window
                before = min(sinks, base) + max(0, base - max(old, sinks, 0))
                hidden = max(0, old - max(base, sinks)) if not c["tree"] else 0
                seen += before + max(0, o - hidden)
        bytes_ = 2 * read * c["Hkv"] * c["D"] * e + sum(windows) * c["Hq"] * (2 * c["D"] * e + 4)
        return {"bytes": bytes_, "flops": 4 * c["D"] * c["Hq"] * seen}
    if c["op"] == "verify":
        small = 4 * (2 * sum(_windows(c)) + 2 * c["B"] * c["N"] + 2 * c["B"])
        rows = sum(len(p) for p in _paths(c))
        if c["tokens"]:
            return {"bytes": small + 4 * rows, "flops": sum(_windows(c))}
        return {"bytes": small + rows * c["V"] * e, "flops": (1 if c["greedy"] else 4) * rows * c["V"]}
    per = 2 * 2 * c["layers"] * c["Hkv"] * c["D"] * e                        # a token's keys and values, read and written
    if c["op"] == "compact":
        moved = sum(1 for p in _paths(c) for i, x in enumerate(p) if i != x)
        return {"bytes": moved * per + 4 * (sum(len(p) for p in _paths(c)) + 4 * c["B"]), "flops": 0}
    return {"bytes": sum(_used(c)) * per + 8 * c["M"], "flops": 0}


# --------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# --------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "verify":
        return None                                                            # whole numbers only
    s = prepare(case, seed)
    return {"attend": _exact_attend, "compact": _exact_compact, "copy": _exact_copy}[case["op"]](s)


def _exact_attend(s):
    B, N, Hq, D = s["q"].shape
    G, page, W, sinks = Hq // s["Hkv"], s["page"], s["window"], s["sinks"]
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    parents, depths = _trees(s) if s["tree"] else (None, None)
    for b, (L, n) in enumerate(zip(_kv_lens(s), _windows(s))):
        if n == 0:
            continue
        base = L - n
        cut = base - W + 1 if W else 0                                         # nobody sees what is older, but for the sinks
        kept = [x for x in range(min(sinks, L)) if x < cut] + list(range(max(cut, 0), L)) if W else list(range(L))
        j = torch.tensor(kept, device="cuda")
        seen = torch.empty(n, len(kept), dtype=torch.bool, device="cuda")
        for i in range(n):
            if s["tree"]:
                row, at = j < base, i
                while at >= 0:
                    row = row | (j == base + at)
                    at = parents[b][at]
                p = base + depths[b][i]
            else:
                p = base + i
                row = j <= p if s["causal"] else j < L
            if W:
                row = row & ((j < sinks) | (j > p - W))
            seen[i] = row
        pages = s["block_table"][b].long()[j // page]
        for h in range(s["Hkv"]):
            k, v = s["k_cache"][pages, h, j % page].double(), s["v_cache"][pages, h, j % page].double()
            for g in range(h * G, (h + 1) * G):
                z = (s["q"][b, :n, g].double() @ k.T * s["scale"]).masked_fill_(~seen, -math.inf)
                total = torch.logsumexp(z, dim=-1, keepdim=True)
                out[b, :n, g] = z.sub_(total).exp_() @ v
                lse[b, :n, g] = total[:, 0]
    return {"out": out, "lse": lse}


def _exact_compact(s):
    lens, page = _kv_lens(s), s["page"]
    table = s["block_table"].tolist()
    kv_len, src, dst = [], [], []
    for b, (L, n, path) in enumerate(zip(lens, _windows(s), _paths(s))):
        kv_len.append(L - n + len(path))
        for i, x in enumerate(path):
            for at, places in ((L - n + x, src), (L - n + i, dst)):
                places.append(table[b][at // page] * page + at % page)
    src, dst = (torch.tensor(x, dtype=torch.long, device="cuda") for x in (src, dst))
    caches = []
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.double().transpose(2, 3).flatten(1, 2)                    # [layers, slots, Hkv, D]
        flat[:, dst] = flat[:, src]
        caches.append(flat.view(cache.shape[0], -1, page, s["Hkv"], s["D"]).transpose(2, 3))
    return {"kv_len": None, "k_cache": caches[0], "v_cache": caches[1]}


def _exact_copy(s):
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for x, y, used in zip(s["src"].tolist(), s["dst"].tolist(), _used(s)):
        for cache in caches:
            cache[:, y, :, :used] = cache[:, x, :, :used]
    return dict(zip(("k_cache", "v_cache"), caches))
