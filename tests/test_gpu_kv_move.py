"""GPU parity: moving the accepted path's keys and values together, and copying pages; bit for bit."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


def _bits(shape, seed, dtype="bf16"):
    """Caches of any 16 bits, NaN among them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int16)
    return x.view(torch.bfloat16 if dtype == "bf16" else torch.float16)


def _ints(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _host(t):
    import torch
    return t.view(torch.int16).cpu().numpy()


class CompactCase:
    def __init__(self, layers, Hkv, page, D, kv_len, N, lengths=None, seed=0, dtype="bf16", paths=None):
        rng = np.random.default_rng(seed)
        B = len(kv_len)
        need = [-(-L // page) for L in kv_len]
        P = sum(need) + 2
        order = rng.permutation(P)
        self.table = np.full((B, max(max(need), 1) + 1), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.kv_len, self.N, self.page = np.asarray(kv_len, np.int32), N, page
        self.lengths = None if lengths is None else np.asarray(lengths, np.int32)
        self.path, self.accepted = np.full((B, N), -1, np.int32), np.zeros(B, np.int32)
        for b in range(B):
            n = self.n(b)
            if n == 0:
                continue
            p = paths[b] if paths else [0] + sorted((1 + rng.permutation(n - 1)[:rng.integers(0, n)]).tolist())
            self.path[b, :len(p)], self.accepted[b] = p, len(p) - 1
        shape = (layers, P, Hkv, page, D)
        self.k, self.v = _bits(shape, seed, dtype), _bits(shape, seed + 1, dtype)

    def n(self, b):
        return self.N if self.lengths is None else int(self.lengths[b])

    def expected(self):
        k, v, out = _host(self.k), _host(self.v), []
        for b in range(len(self.kv_len)):
            args = (self.table[b].tolist(), int(self.kv_len[b]), self.n(b), self.path[b].tolist(), int(self.accepted[b]))
            k, length = oracle.compact(k, *args)
            v, _ = oracle.compact(v, *args)
            out.append(length)
        return k, v, out

    def run(self, ds, **kw):
        return ds.dspark_kv_compact(self.k, self.v, _ints(self.table), _ints(self.kv_len), _ints(self.path), _ints(self.accepted),
                                    lengths=None if self.lengths is None else _ints(self.lengths), **kw)

    def check(self, ds, **kw):
        k, v, lens = self.expected()
        out = self.run(ds, **kw)
        assert out.tolist() == lens
        np.testing.assert_array_equal(_host(self.k), k)
        np.testing.assert_array_equal(_host(self.v), v)


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("Hkv,page,D", [(1, 1, 8), (2, 16, 64), (8, 16, 128), (3, 7, 24), (1, 256, 512), (5, 8, 72)])
@pytest.mark.parametrize("N", [1, 2, 9, 33, 256])
def test_compact_shapes(cuda_lib, layers, Hkv, page, D, N):
    lens = [N, N + 1, N + page, N + 2 * page + 3]
    CompactCase(layers, Hkv, page, D, lens, N, seed=N + page, dtype="f16" if N % 2 else "bf16").check(cuda_lib)


def test_compact_ragged_requests(cuda_lib):
    case = CompactCase(2, 2, 16, 64, [0, 5, 40, 40, 33, 100], 8, lengths=[0, 5, 0, 8, 1, 7], seed=3)
    case.check(cuda_lib)
    before = _host(case.k).copy()
    case.kv_len[2] = 40                                       # nothing to move: nothing is written
    case.path[:, 1:], case.accepted[:] = -1, 0
    case.check(cuda_lib)
    np.testing.assert_array_equal(_host(case.k), before)


def test_compact_full_paths_and_every_shift(cuda_lib):
    N = 40
    paths = [list(range(N)), [0, N - 1], list(range(0, N, 2)), [0] + list(range(N - 9, N)), list(range(1, N)), [5], list(range(8, N))]
    CompactCase(2, 2, 16, 64, [N + 13 * b for b in range(len(paths))], N, paths=paths, seed=5).check(cuda_lib)


def test_compact_many_requests(cuda_lib):
    rng = np.random.default_rng(7)
    N = rng.integers(0, 13, 3000)
    CompactCase(1, 1, 8, 16, (N + rng.integers(0, 30, 3000)).tolist(), 12, lengths=N, seed=7).check(cuda_lib)


def test_compact_more_requests_than_a_grid_is_high(cuda_lib):
    import torch
    B = 65535 + 700
    case = CompactCase(1, 1, 4, 8, [4] * 3, 4, seed=9)
    k = _bits((1, B, 1, 4, 8), 1)
    v = k.clone()
    want = k.clone()
    want[:, :, :, 1] = k[:, :, :, 3]
    path = torch.tensor([[0, 3, -1, -1]], dtype=torch.int32, device="cuda").repeat(B, 1)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    full = lambda x: torch.full((B,), x, dtype=torch.int32, device="cuda")
    out = cuda_lib.dspark_kv_compact(k, v, table, full(4), path, full(1))
    assert bool((out == 2).all()) and np.array_equal(_host(k), _host(want)) and np.array_equal(_host(v), _host(want))


def test_compact_flags_what_is_out_of_range(cuda_lib):
    ds = cuda_lib
    ws = ds.Workspace(ds.OP_KV_COMPACT)
    ws.buf.fill_(255)

    def fresh():
        return CompactCase(2, 2, 16, 64, [60, 50, 40], 8, seed=11, paths=[[0, 2, 5], [0, 3], [0, 1, 4, 7]])

    fresh().check(ds, workspace=ws)
    assert ds.dspark_read_status(ws) == (0, 0)
    for change in (lambda c: c.kv_len.__setitem__(1, 7), lambda c: c.kv_len.__setitem__(1, 10 ** 6), lambda c: c.kv_len.__setitem__(1, -5),
                   lambda c: c.accepted.__setitem__(1, 8), lambda c: c.accepted.__setitem__(1, -1),
                   lambda c: c.path.__setitem__((1, 1), 0), lambda c: c.path.__setitem__((1, 1), 8), lambda c: c.path.__setitem__((1, 1), -1),
                   lambda c: c.path.__setitem__((1, 0), -1), lambda c: c.path.__setitem__((1, 0), 2 ** 31 - 1)):
        case, clean = fresh(), fresh()
        change(case)
        clean.accepted[1], clean.path[1] = 7, range(8)        # request 1 as if it kept everything
        k, v, lens = clean.expected()
        lens[1] = int(case.kv_len[1])
        out = case.run(ds, workspace=ws)
        assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE and out.tolist() == lens
        np.testing.assert_array_equal(_host(case.k), k)
        np.testing.assert_array_equal(_host(case.v), v)
    for value in (9, -1):
        case = fresh()
        case.lengths = np.array([8, value, 8], np.int32)
        out = case.run(ds, workspace=ws)
        assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE and out.tolist() == [55, 50, 36]
    case = fresh()
    case.table[0, (52 + 5) // 16] = 10 ** 6                   # the page of a source: that token stays, the others move
    want = fresh()
    out = case.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws)[1] & ds.STATUS_INPUT_RANGE and out.tolist() == want.expected()[2]


def test_caches_within_a_larger_pool(cuda_lib):
    """Layers that are far apart: the memory between them stays as it is."""
    import torch
    case = CompactCase(3, 2, 16, 64, [60, 50], 8, seed=13)
    k, v, lens = case.expected()
    P = case.k.shape[1]
    for name in ("k", "v"):
        pool = _bits((3, P + 4, 2, 16, 64), 99)
        pool[:, :P] = getattr(case, name)
        setattr(case, name + "_pool", pool)
        setattr(case, name, pool[:, :P])
    rest = _host(case.k_pool)[:, P:].copy()
    assert case.run(cuda_lib).tolist() == lens
    np.testing.assert_array_equal(_host(case.k_pool)[:, :P], k)
    np.testing.assert_array_equal(_host(case.v_pool)[:, :P], v)
    np.testing.assert_array_equal(_host(case.k_pool)[:, P:], rest)
    cuda_lib.dspark_kv_copy_pages(case.k, case.v, _ints([1, 2]), _ints([0, 3]), used=_ints([16, 3]))
    np.testing.assert_array_equal(_host(case.k_pool)[:, :P], oracle.copy_pages(k, [1, 2], [0, 3], [16, 3]))
    np.testing.assert_array_equal(_host(case.k_pool)[:, P:], rest)


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("Hkv,page,D", [(1, 1, 8), (2, 16, 64), (8, 16, 128), (3, 7, 24), (1, 256, 512), (16, 128, 128)])
def test_copy_shapes(cuda_lib, layers, Hkv, page, D):
    rng = np.random.default_rng(page)
    P = 14
    k, v = _bits((layers, P, Hkv, page, D), 1), _bits((layers, P, Hkv, page, D), 2)
    order = rng.permutation(P)
    dst, src = order[:6], rng.choice(order[6:], 6)            # sources more than once
    for used in (None, rng.integers(0, page + 1, 6)):
        want = [oracle.copy_pages(_host(c), src, dst, used) for c in (k, v)]
        cuda_lib.dspark_kv_copy_pages(k, v, _ints(src), _ints(dst), used=None if used is None else _ints(used))
        for c, w in zip((k, v), want):
            np.testing.assert_array_equal(_host(c), w)
        k, v = _bits((layers, P, Hkv, page, D), 3), _bits((layers, P, Hkv, page, D), 4)


def test_copy_many_pages_one_cache_and_itself(cuda_lib):
    import torch
    P = 5000
    k, v = _bits((P, 1, 8, 16), 1), _bits((P, 1, 8, 16), 2)
    order = np.random.default_rng(0).permutation(P)
    src, dst = np.concatenate([order[:2000], [order[0]]]), np.concatenate([order[2000:4000], [order[0]]])
    want = [oracle.copy_pages(_host(c)[None], src, dst)[0] for c in (k, v)]
    cuda_lib.dspark_kv_copy_pages(k, v, _ints(src), _ints(dst))
    for c, w in zip((k, v), want):
        np.testing.assert_array_equal(_host(c), w)


def test_copy_flags_what_is_out_of_range(cuda_lib):
    ds = cuda_lib
    ws = ds.Workspace(ds.OP_KV_COPY_PAGES)
    ws.buf.fill_(255)
    for bad in (dict(src=8), dict(src=-1), dict(dst=8), dict(dst=-1), dict(used=17), dict(used=-1), {}):
        k, v = _bits((2, 8, 2, 16, 64), 1), _bits((2, 8, 2, 16, 64), 2)
        src, dst, used = [0, 1, 2], [3, 4, 5], [16, 9, 2]
        for name, x in (("src", src), ("dst", dst), ("used", used)):
            x[1] = bad.get(name, x[1])
        keep = [0, 2] if bad else [0, 1, 2]
        want = [oracle.copy_pages(_host(c), [src[i] for i in keep], [dst[i] for i in keep], [used[i] for i in keep]) for c in (k, v)]
        ds.dspark_kv_copy_pages(k, v, _ints(src), _ints(dst), used=_ints(used), workspace=ws)
        assert ds.dspark_read_status(ws)[1] == (ds.STATUS_INPUT_RANGE if bad else 0)
        for c, w in zip((k, v), want):
            np.testing.assert_array_equal(_host(c), w)


def test_capture_and_another_stream(cuda_lib):
    import torch
    case = CompactCase(2, 2, 16, 64, [60, 50], 8, seed=17)
    k, v, lens = case.expected()
    start = [case.k.clone(), case.v.clone()]
    ws, ws2 = cuda_lib.Workspace(cuda_lib.OP_KV_COMPACT), cuda_lib.Workspace(cuda_lib.OP_KV_COPY_PAGES)
    args = [_ints(x) for x in (case.table, case.kv_len, case.path, case.accepted)]
    out, src, dst = torch.empty(2, dtype=torch.int32, device="cuda"), _ints([int(case.table[0, 0])]), _ints([int(case.table[1, 0])])

    def call():
        cuda_lib.dspark_kv_compact(case.k, case.v, *args, kv_len_out=out, workspace=ws)
        cuda_lib.dspark_kv_copy_pages(case.k, case.v, src, dst, workspace=ws2)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    case.k.copy_(start[0])
    case.v.copy_(start[1])
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert out.tolist() == lens
    for c, w in ((case.k, k), (case.v, v)):
        np.testing.assert_array_equal(_host(c), oracle.copy_pages(w, src.tolist(), dst.tolist()))


def test_offsets_past_32_bits(cuda_lib):
    import torch
    P = (1 << 31) // (8 * 64 * 128) + 40
    k = torch.zeros(1, P, 8, 64, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = CompactCase(1, 8, 64, 128, [200], 30, seed=19)
    n = 4
    for dst, src in ((k, small.k), (v, small.v)):
        dst[:, P - n:] = src[:, small.table[0, :n]]
    table = torch.arange(P - n, P, dtype=torch.int32, device="cuda")[None].contiguous()
    wk, wv, lens = small.expected()
    out = cuda_lib.dspark_kv_compact(k, v, table, _ints([200]), _ints(small.path), _ints(small.accepted))
    assert out.tolist() == lens
    np.testing.assert_array_equal(_host(k[:, P - n:]), wk[:, small.table[0, :n]])
    np.testing.assert_array_equal(_host(v[:, P - n:]), wv[:, small.table[0, :n]])
    cuda_lib.dspark_kv_copy_pages(k, v, _ints([P - 1]), _ints([0]))
    assert torch.equal(k[:, 0].view(torch.int16), k[:, P - 1].view(torch.int16))


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    c = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    k = c(4, 2, 16, 64)
    lens = i(1)
    good = lambda k=k, v=k, table=i(1, 2), kv=lens, path=i(1, 3) - 1, acc=i(1), **kw: ds.dspark_kv_compact(k, v, table, kv, path, acc, **kw)
    for bad in (dict(k=k.float(), v=k.float()), dict(table=i(1, 2).long()), dict(path=c(1, 3))):
        with pytest.raises(TypeError):
            good(**bad)
    for bad in (dict(k=k.transpose(0, 1)), dict(k=k[0], v=k[0]), dict(v=c(4, 2, 16, 32)), dict(v=k.half()), dict(acc=i(2)), dict(table=i(2, 2)),
                dict(lengths=i(2)), dict(kv_len_out=i(2)), dict(k=c(2, 6, 2, 16, 64)[:, :4], v=c(2, 4, 2, 16, 64))):
        with pytest.raises(ValueError):
            good(**bad)
    for bad in (dict(kv_len_out=lens), dict(path=i(1, 257))):
        with pytest.raises(ds.DSparkError) as e:
            good(**bad)
        assert e.value.status == 1
    for bad in ((k, k, i(2), i(3)), (k, k, i(2), i(2), i(3))):
        with pytest.raises(ValueError):
            ds.dspark_kv_copy_pages(*bad)
    with pytest.raises(ds.DSparkError):
        ds.dspark_kv_copy_pages(k, k, i(0), i(0))
