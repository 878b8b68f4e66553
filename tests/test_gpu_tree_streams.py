"""The tree operators on a given stream: what a call allocates belongs to it, and two calls at once on two streams, each
with its own workspace, come to what they come to alone."""
import numpy as np
import pytest

from tests._trees import TreeCase, WindowCase, random_parents
from tests.test_gpu_kv_move import CompactCase, _bits, _ints
from tests.test_gpu_verify_tree import VerifyCase

pytestmark = pytest.mark.gpu

NAMES = ["tree_attention", "window_attention", "verify_tree", "verify_tree_tokens", "kv_compact", "kv_copy_pages"]


def _calls(ds, seed=0):
    """name -> a function of (stream, workspace) that makes the call and returns its outputs and what it wrote in place."""
    import torch
    rng = np.random.default_rng(seed)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    tree = TreeCase(3, 40, 16, 4, 128, 16, [3000, 1200, 77], parents=random_parents(rng, 3, 40), seed=seed)
    window = WindowCase(3, 5, 16, 4, 64, 32, [3000, 1200, 77], "f16", seed=seed, window=500, sinks=4)
    verify = VerifyCase(9, 12, 30011, seed=seed)
    compact = CompactCase(3, 2, 16, 64, [60, 50, 33], 20, seed=seed)
    target = dev(rng.integers(0, 5, (9, 12)).astype(np.int32))
    draft = dev(rng.integers(0, 5, (9, 12)).astype(np.int32))
    parents = dev(verify.parents)
    t = [dev(x) for x in (tree.table, tree.kv_len, tree.parents)]
    w = [dev(x) for x in (window.table, window.kv_len)]
    v = [dev(x) for x in (verify.tokens, verify.T, verify.u)]
    c = [_ints(x) for x in (compact.table, compact.kv_len, compact.path, compact.accepted)]
    k, vv, src, dst = _bits((2, 9, 2, 16, 64), 1), _bits((2, 9, 2, 16, 64), 2), _ints([1, 1, 2]), _ints([5, 6, 7])

    def moved(caches, call):
        def run(stream, ws):
            with torch.cuda.stream(stream):
                own = [x.clone() for x in caches]
            out = call(*own, stream, ws)
            return [out] * (out is not None) + own
        return run

    return {
        "tree_attention": lambda s, ws: [ds.dspark_tree_attention(tree.q, tree.k, tree.v, *t, tree.scale, workspace=ws, stream=s)],
        "window_attention": lambda s, ws: [ds.dspark_window_attention(window.q, window.k, window.v, *w, 500, 4, window.scale,
                                                                     workspace=ws, stream=s)],
        "verify_tree": lambda s, ws: list(ds.dspark_verify_tree(verify.target, parents, *v, workspace=ws, stream=s)),
        "verify_tree_tokens": lambda s, ws: list(ds.dspark_verify_tree_tokens(target, parents, draft, workspace=ws, stream=s)),
        "kv_compact": moved((compact.k, compact.v), lambda a, b, s, ws: ds.dspark_kv_compact(a, b, *c, workspace=ws, stream=s)),
        "kv_copy_pages": moved((k, vv), lambda a, b, s, ws: ds.dspark_kv_copy_pages(a, b, src, dst, workspace=ws, stream=s)),
    }


def _same(a, b):
    import torch
    bits = lambda x: x.view(torch.int16) if x.element_size() == 2 else x
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_given_stream(cuda_lib, name, monkeypatch):
    import torch
    call = _calls(cuda_lib)[name]
    want = call(torch.cuda.current_stream(), None)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []
    for maker in ("empty", "empty_like"):
        plain = getattr(torch, maker)

        def recorded(*a, plain=plain, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return plain(*a, **kw)

        monkeypatch.setattr(torch, maker, recorded)
    got = call(other, None)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert seen and all(s == other.cuda_stream for s in seen)
    assert _same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(cuda_lib, name):
    import torch
    ds = cuda_lib
    calls = [_calls(ds, seed)[name] for seed in (0, 1)]
    want = [c(torch.cuda.current_stream(), None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    sizes = {"tree_attention": (ds.OP_TREE_ATTENTION, 3, 40, 16, 128), "window_attention": (ds.OP_WINDOW_ATTENTION, 3, 5, 16, 64),
             "verify_tree": (ds.OP_VERIFY_TREE,), "verify_tree_tokens": (ds.OP_VERIFY_TREE,), "kv_compact": (ds.OP_KV_COMPACT,),
             "kv_copy_pages": (ds.OP_KV_COPY_PAGES,)}[name]
    spaces = [ds.Workspace(*sizes) for _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        got = [c(s, ws) for c, s, ws in zip(calls, streams, spaces)]
    torch.cuda.synchronize()
    for g, w, ws in zip(got, want, spaces):
        assert _same(g, w) and ds.dspark_read_status(ws) == (0, 0)


def test_a_captured_round_of_all_of_them(cuda_lib):
    """Verification, compaction, a page's copy and the next attention in one graph, replayed on new inputs."""
    import torch
    ds = cuda_lib
    B, N, V, Hkv, D, page = 3, 12, 5003, 2, 64, 16
    rng = np.random.default_rng(0)
    case = TreeCase(B, N, 8, Hkv, D, page, [200, 77, 40], parents=random_parents(rng, B, N), seed=1)
    vc = VerifyCase(B, N, V, seed=2)
    vc.parents = case.parents
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    table, kv, parents, tokens, T, u = (dev(x) for x in (case.table, case.kv_len, case.parents, vc.tokens, vc.T, vc.u))
    k, v = case.k.clone(), case.v.clone()
    spaces = [ds.Workspace(ds.OP_VERIFY_TREE), ds.Workspace(ds.OP_KV_COMPACT), ds.Workspace(ds.OP_KV_COPY_PAGES),
              ds.Workspace(ds.OP_TREE_ATTENTION, B, N, 8, D)]
    outs = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B, N), (B,))]
    spare = sorted(set(range(case.k.shape[0])) - set(case.table.flatten().tolist()))[0]
    src, dst = _ints([int(case.table[0, 0])]), _ints([spare])
    attended = torch.empty_like(case.q)

    def round_(k, v, outs, attended, spaces):
        ds.dspark_verify_tree(vc.target, parents, tokens, T, u, None, *outs[:3], workspace=spaces[0])
        ds.dspark_kv_compact(k, v, table, kv, outs[2], outs[1], kv_len_out=outs[3], workspace=spaces[1])
        ds.dspark_kv_copy_pages(k, v, src, dst, workspace=spaces[2])
        ds.dspark_tree_attention(case.q, k, v, table, kv, parents, case.scale, out=attended, workspace=spaces[3])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        round_(k, v, outs, attended, spaces)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        round_(k, v, outs, attended, spaces)
    for seed in (3, 4, 5):
        u.copy_(torch.from_numpy(np.random.default_rng(seed).random((B, N)).astype(np.float32)))
        T.fill_(0.5 * (seed - 3))
        k.copy_(case.k)
        v.copy_(case.v)
        g.replay()
        torch.cuda.synchronize()
        eager = [torch.empty_like(x) for x in outs]
        ek, ev, ea = case.k.clone(), case.v.clone(), torch.empty_like(attended)
        round_(ek, ev, eager, ea, [None] * 4)
        assert _same(outs + [k, v, attended], eager + [ek, ev, ea])
        assert all(ds.dspark_read_status(ws) == (0, 0) for ws in spaces)
