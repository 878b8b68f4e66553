"""GPU parity: verification of drafted trees, token for token against the integer oracle on the device's own weights."""
import math

import numpy as np
import pytest

import oracle
from oracle.sample import MASS
from tests._trees import random_parents
from tests.test_gpu_sample import _weights

pytestmark = pytest.mark.gpu


class VerifyCase:
    """Trees with target logits that follow a path of each for a while."""

    def __init__(self, B, N, V, seed=0, bf16=False, greedy=False, lengths=None, shape="random", follow=0.85, gain=3.0):
        import torch
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.N, self.V = B, N, V
        self.parents = random_parents(rng, B, N, deepest=12 if shape == "random" else None, shape=shape)
        self.tokens = rng.integers(0, V, (B, N)).astype(np.int32)
        x = torch.randn(B, N, V, generator=g, device="cuda") * gain
        for b in range(B):
            for i in range(1, N):                             # the last child so treated is the one that counts
                p = int(self.parents[b, i])
                if p >= 0 and rng.random() < follow:
                    x[b, p, int(self.tokens[b, i])] = 25.0 + 0.5 * (i % 7)
        self.target = x.to(torch.bfloat16) if bf16 else x
        self.lengths = None if lengths is None else np.asarray(lengths, np.int32)
        self.T = None if greedy else rng.choice([0.0, 0.5, 0.8, 1.0, 3.0], B).astype(np.float32)
        self.u = None if greedy else rng.random((B, N)).astype(np.float32)

    def run(self, ds, **kw):
        import torch
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()
        out = ds.dspark_verify_tree(self.target, dev(self.parents), dev(self.tokens), dev(self.T), dev(self.u), dev(self.lengths), **kw)
        return [t.cpu().numpy() for t in out]

    def expected(self):
        out = np.full((self.B, self.N), -1, np.int32)
        path, accepted = out.copy(), np.zeros(self.B, np.int32)
        for b in range(self.B):
            n = self.N if self.lengths is None else int(self.lengths[b])
            T = 0.0 if self.T is None else float(self.T[b])

            def token(node):
                import torch
                x = self.target[b, node].float()[None]
                w = _weights(x, torch.tensor([T], device="cuda"))[0].cpu().numpy().astype(np.float64)
                x = x[0].cpu().numpy()
                if not np.isfinite(x).any():
                    return 0
                if T == 0:
                    return int(np.argmax(np.where(np.isfinite(x), x, -np.inf)))
                mass = np.floor(w * MASS).astype(np.uint64)   # below 2^61 in all
                t = int(mass.sum()) * int(math.floor(float(self.u[b, node]) * 2 ** 24)) >> 24
                return int(np.searchsorted(np.cumsum(mass), np.uint64(t), side="right"))

            tok, p = oracle.verify_tree(token, self.parents[b].tolist(), self.tokens[b].tolist(), n)
            out[b, :len(tok)], path[b, :len(p)], accepted[b] = tok, p, max(0, len(p) - 1)
        return out, accepted, path

    def check(self, ds, **kw):
        got = self.run(ds, **kw)
        for name, a, z in zip(("tokens", "accepted", "path"), got, self.expected()):
            np.testing.assert_array_equal(a, z, err_msg=name)
        return got


def test_the_oracle_s_draw_is_the_sampling_oracle_s(cuda_lib):
    import torch
    rng = np.random.default_rng(0)
    x = rng.standard_normal(50) * 3
    w = _weights(torch.tensor(x[None], dtype=torch.float32, device="cuda"), torch.tensor([0.8], device="cuda"))[0].cpu().numpy()
    for u in rng.random(20).astype(np.float32):
        mass = np.floor(w.astype(np.float64) * MASS).astype(np.uint64)
        t = int(mass.sum()) * int(math.floor(float(u) * 2 ** 24)) >> 24
        assert oracle.tree_token(x, w, 0.8, u) == int(np.searchsorted(np.cumsum(mass), np.uint64(t), side="right"))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 33, 1000, 1023, 4097, 50001, 151936])
def test_vocabularies_and_types(cuda_lib, V, bf16):
    B, N = (6, 9) if V < 10000 else (3, 7)
    VerifyCase(B, N, V, seed=V, bf16=bf16).check(cuda_lib)
    VerifyCase(B, N, V, seed=V + 1, bf16=bf16, greedy=True).check(cuda_lib)


@pytest.mark.parametrize("B", [1, 2, 5, 9, 10, 19, 38, 39, 76, 77, 152, 153, 305, 700])
def test_request_counts(cuda_lib, B):
    """Every number of blocks per request, and more requests than blocks at once."""
    VerifyCase(B, 6, 20011, seed=B).check(cuda_lib)


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 200, 256])
@pytest.mark.parametrize("shape", ["random", "chain", "star", "forest"])
def test_trees(cuda_lib, N, shape):
    VerifyCase(4, N, 701, seed=N, shape=shape, follow=0.97).check(cuda_lib)


def test_a_chain_accepted_to_its_end(cuda_lib):
    case = VerifyCase(2, 256, 3000, seed=5, shape="chain", follow=1.0, greedy=True)
    out, accepted, path = case.check(cuda_lib)
    assert accepted.tolist() == [255, 255] and path[0].tolist() == list(range(256)) and (out >= 0).all()


def test_lengths_and_padding(cuda_lib):
    case = VerifyCase(6, 10, 999, seed=7, lengths=[0, 1, 10, 5, 0, 2], follow=1.0)
    out, accepted, path = case.check(cuda_lib)
    assert (out[0] == -1).all() and (path[0] == -1).all() and accepted[0] == 0 and path[1].tolist() == [0] + [-1] * 9


def test_uniforms_at_the_ends_and_equal_logits(cuda_lib):
    import torch
    case = VerifyCase(8, 4, 5003, seed=9, follow=0.0)
    case.T[:] = 1.0
    case.u[:] = np.array([0.0, 1.0 - 2.0 ** -24, 2.0 ** -24, 0.5], np.float32)
    case.check(cuda_lib)
    case.target.fill_(1.5)                                    # every mass is 2^40
    case.u[:, 0] = np.linspace(0, 1 - 2.0 ** -24, 8, dtype=np.float32)
    out = case.check(cuda_lib)[0]
    assert out[0, 0] == 0 and out[7, 0] == 5002
    case.target[:] = -math.inf
    case.target[:, :, 77] = -3.0                              # a single unmasked entry, and two
    assert (case.check(cuda_lib)[0][:, 0] == 77).all()
    case.target[:, :, 5001] = -3.0
    case.check(cuda_lib)
    case.T[:] = 1e-45                                         # 1 / T overflows: entries equal to the largest share the mass
    case.target[:, :, 10] = -3.0000002
    case.check(cuda_lib)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [997, 30011, 151936])
def test_draws_at_the_ends_of_entries(cuda_lib, V, bf16):
    """Uniforms whose share of the mass is an entry's first unit, its last, or next to them: sums in fp32 cannot tell."""
    import torch
    case = VerifyCase(24, 1, V, seed=V, bf16=bf16, follow=0.0)
    case.T[:] = np.tile([0.6, 1.0, 2.5], 8).astype(np.float32)
    w = _weights(case.target[:, 0].float(), torch.from_numpy(case.T).cuda()).cpu().numpy().astype(np.float64)
    rng = np.random.default_rng(1)
    for b in range(24):
        mass = np.floor(w[b] * MASS).astype(np.uint64)
        ends = np.cumsum(mass)
        v = int(np.searchsorted(ends, np.uint64(int(rng.integers(0, int(ends[-1])))), side="right"))
        # the smallest uniform that is past entry v - 1, and its neighbours
        u = -(-int(ends[v] - mass[v]) * 2 ** 24 // int(ends[-1])) + b % 3 - 1
        case.u[b, 0] = min(max(u, 0), 2 ** 24 - 1) * 2.0 ** -24
    case.check(cuda_lib)


@pytest.mark.parametrize("T", [0.01, 0.1, 30.0, 1e4])
@pytest.mark.parametrize("gain", [0.01, 3.0, 100.0, 1e6])
def test_scales_of_logits_and_temperatures(cuda_lib, T, gain):
    import torch
    case = VerifyCase(8, 3, 20011, seed=21, follow=0.0, gain=gain)
    case.T[:] = T
    case.check(cuda_lib)
    case.target += 1e5                                        # far from 0, where a shift loses bits
    case.check(cuda_lib)
    case.target[:, :, :700] = -math.inf                       # nothing to go by among the first entries
    case.check(cuda_lib)


@pytest.mark.parametrize("B", [1, 40, 700])
def test_odd_values_in_rows_that_are_drawn_from(cuda_lib, B):
    import torch
    case = VerifyCase(B, 2, 5003, seed=B, follow=0.0)
    case.T[:] = 1.0
    ws = cuda_lib.Workspace(cuda_lib.OP_VERIFY_TREE, B, 2)
    for at in (0, 1, 2500, 5002):
        for value in (math.nan, math.inf):
            case.target[::2, 0, at] = value
            case.check(cuda_lib, workspace=ws)
            assert cuda_lib.dspark_read_status(ws)[1] == cuda_lib.STATUS_NUMERIC


def test_ties_go_to_the_lowest_id(cuda_lib):
    import torch
    case = VerifyCase(3, 3, 40009, seed=11, greedy=True, follow=0.0)
    for at in ([5, 40008], [0, 1], [20000, 20001, 39999]):
        case.target[:] = torch.randn_like(case.target)
        for v in at:
            case.target[:, :, v] = 9.0
        assert (case.check(cuda_lib)[0][:, 0] == at[0]).all()
    case.target[:] = -0.0
    case.target[:, :, 30] = 0.0                               # -0 equals +0
    assert (case.check(cuda_lib)[0][:, 0] == 0).all()


def test_equals_sampling_all_nodes_first(cuda_lib):
    """The same tokens as dspark_sample draws for every node, walked by dspark_verify_tree_tokens."""
    import torch
    ds = cuda_lib
    case = VerifyCase(20, 12, 30011, seed=13)
    R = 20 * 12
    col = lambda x, t=torch.float32: torch.full((R,), x, dtype=t, device="cuda")
    T, u = torch.from_numpy(case.T).cuda().repeat_interleave(12), torch.from_numpy(case.u).cuda().flatten()
    tokens = ds.dspark_sample(case.target.view(R, -1), T, col(0, torch.int32), col(1.0), col(0.0), u).view(20, 12)
    dev = lambda x: torch.from_numpy(x).cuda()
    walked = ds.dspark_verify_tree_tokens(tokens, dev(case.parents), dev(case.tokens))
    for a, z in zip(walked, case.check(ds)):
        np.testing.assert_array_equal(a.cpu().numpy(), z)


@pytest.mark.parametrize("B,N", [(1, 1), (1, 256), (3, 33), (64, 64), (65, 7), (3000, 20)])
@pytest.mark.parametrize("shape", ["random", "chain", "forest"])
def test_tokens_given(cuda_lib, B, N, shape):
    import torch
    rng = np.random.default_rng(B + N)
    parents = random_parents(rng, B, N, shape=shape)
    draft, target = rng.integers(0, 4, (B, N)).astype(np.int32), rng.integers(0, 4, (B, N)).astype(np.int32)
    lengths = rng.integers(0, N + 1, B).astype(np.int32)
    dev = lambda x: torch.from_numpy(x).cuda()
    for ln in (None, lengths):
        got = cuda_lib.dspark_verify_tree_tokens(dev(target), dev(parents), dev(draft), None if ln is None else dev(ln))
        out, accepted, path = [t.cpu().numpy() for t in got]
        for b in range(B):
            n = N if ln is None else int(ln[b])
            tok, p = oracle.verify_tree(lambda i: int(target[b, i]), parents[b].tolist(), draft[b].tolist(), n)
            assert out[b].tolist() == tok + [-1] * (N - len(tok)) and path[b].tolist() == p + [-1] * (N - len(p))
            assert accepted[b] == max(0, len(p) - 1)


def test_device_side_checks(cuda_lib):
    import torch
    ds = cuda_lib
    ws = ds.Workspace(ds.OP_VERIFY_TREE, 4, 6)
    case = VerifyCase(4, 6, 500, seed=17, follow=1.0)
    case.T[:] = [0.0, 1.0, 0.7, 1.0]
    clean = case.check(ds, workspace=ws)
    assert ds.dspark_read_status(ws) == (0, 0)

    def flagged(bit):
        got = case.run(ds, workspace=ws)
        assert ds.dspark_read_status(ws)[1] == bit
        return got

    case.lengths = np.array([6, 7, -1, 6], np.int32)
    out, accepted, path = flagged(ds.STATUS_INPUT_RANGE)
    assert (out[1:3] == -1).all() and (path[1:3] == -1).all() and (accepted[1:3] == 0).all()
    assert np.array_equal(out[0], clean[0][0]) and np.array_equal(out[3], clean[0][3])
    case.lengths = None
    keep = case.parents.copy()
    case.parents[0, 3] = 3
    got = flagged(ds.STATUS_INPUT_RANGE)
    case.parents[0, 3] = -1
    for a, z in zip(got, case.check(ds)):
        np.testing.assert_array_equal(a, z)
    case.parents = keep
    token = int(case.tokens[1, 2])
    for value in (500, -1, 2 ** 31 - 1):
        case.tokens[1, 2] = value
        got = flagged(ds.STATUS_INPUT_RANGE)
        for a, z in zip(got, case.expected()):
            np.testing.assert_array_equal(a, z)
    case.tokens[1, 2] = token
    for value, read in ((1.0, 1.0 - 2.0 ** -24), (-0.5, 0.0), (math.nan, 0.0), (math.inf, 1.0 - 2.0 ** -24)):
        u = case.u.copy()
        case.u[2, 0] = value
        got = flagged(ds.STATUS_INPUT_RANGE)
        case.u[2, 0] = read
        for a, z in zip(got, case.expected()):
            np.testing.assert_array_equal(a, z)
        case.u = u
    for value in (-1.0, math.nan, math.inf):
        case.T[3] = value
        got = flagged(ds.STATUS_NUMERIC)
        case.T[3] = 0.0
        for a, z in zip(got, case.expected()):
            np.testing.assert_array_equal(a, z)
    for value in (math.nan, math.inf):                        # skipped, in the rows that are read
        case.target[0, 0, 3] = value
        got = flagged(ds.STATUS_NUMERIC)
        for a, z in zip(got, case.expected()):
            np.testing.assert_array_equal(a, z)
    case.target[0, 0] = -math.inf
    got = flagged(ds.STATUS_NUMERIC)
    assert got[0][0, 0] == 0
    case.target[0, 0] = 0.0
    unread = next(i for i in range(5, 0, -1) if i not in clean[2][0].tolist())
    case.target[0, unread] = math.nan                         # a row off the path may hold anything
    case.run(ds, workspace=ws)
    bits = ds.dspark_read_status(ws)[1]
    assert bits == (ds.STATUS_NUMERIC if unread in case.expected()[2][0].tolist() else 0)


@pytest.mark.parametrize("B", [1, 30, 200])
def test_capture_replay_streams_and_workspaces(cuda_lib, B):
    import torch
    ds = cuda_lib
    case = VerifyCase(B, 7, 9001, seed=B)
    ws = ds.Workspace(ds.OP_VERIFY_TREE, B, 7)
    ws.buf.fill_(255)
    dev = lambda x: torch.from_numpy(x).cuda()
    parents, tokens, T, u = dev(case.parents), dev(case.tokens), dev(case.T), dev(case.u)
    outs = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B, 7), (B,), (B, 7))]

    def call():
        ds.dspark_verify_tree(case.target, parents, tokens, T, u, None, *outs, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    case.u = np.random.default_rng(5).random((B, 7)).astype(np.float32)
    u.copy_(torch.from_numpy(case.u))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, z in zip(outs, case.expected()):
        np.testing.assert_array_equal(a.cpu().numpy(), z)
    assert ds.dspark_read_status(ws) == (0, 0)


def test_offsets_past_32_bits(cuda_lib):
    import torch
    case = VerifyCase(3, 8, 151936, seed=19, greedy=True, follow=1.0)
    N = 256
    B = (1 << 31) // (N * 151936) + 2                         # more than 2^31 logits
    target = torch.zeros(B, N, 151936, dtype=torch.bfloat16, device="cuda")
    parents = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(B, N, dtype=torch.int32, device="cuda")
    target[B - 1, :8] = case.target[2]
    target[B - 1, 8:] = math.nan
    parents[B - 1, :8] = torch.from_numpy(case.parents[2]).cuda()
    tokens[B - 1, :8] = torch.from_numpy(case.tokens[2]).cuda()
    case.target = case.target.to(torch.bfloat16)
    out, accepted, path = cuda_lib.dspark_verify_tree(target, parents, tokens)
    want = case.expected()
    assert out[B - 1, :8].tolist() == want[0][2].tolist() and int(accepted[B - 1]) == int(want[1][2])
    assert path[B - 1, :8].tolist() == want[2][2].tolist() and (out[:B - 1, 0] == 0).all()


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    x = torch.zeros(2, 3, 10, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    ds.dspark_verify_tree(x, i(2, 3) - 1, i(2, 3))
    for bad in ((x.half(), i(2, 3), i(2, 3)), (x, i(2, 3).long(), i(2, 3)), (x, i(2, 3), f(2, 3)), (x, i(2, 3), i(2, 3), f(2).double(), f(2, 3))):
        with pytest.raises(TypeError):
            ds.dspark_verify_tree(*bad)
    for bad in ((x, i(2, 4), i(2, 4)), (x, i(2, 3), i(2, 4)), (x, i(2, 3), i(2, 3), f(2)), (x, i(2, 3), i(2, 3), f(3), f(2, 3)),
                (x, i(2, 3), i(2, 3), f(2), f(2, 2)), (x, i(2, 3), i(2, 3), None, None, i(3)), (x.transpose(0, 1), i(3, 2), i(3, 2)),
                (x, i(2, 3), i(2, 3), None, None, None, i(2, 4))):
        with pytest.raises(ValueError):
            ds.dspark_verify_tree(*bad)
    with pytest.raises(ValueError):
        ds.dspark_verify_tree_tokens(i(2, 3), i(2, 3), i(2, 4))
    small = ds.Workspace(ds.OP_VERIFY_TREE)
    small.nbytes = 128
    for call in (lambda: ds.dspark_verify_tree(f(1, 257, 4), i(1, 257), i(1, 257)), lambda: ds.dspark_verify_tree(x, i(2, 3), i(2, 3), workspace=small),
                 lambda: ds.dspark_verify_tree_tokens(i(2, 3), i(2, 3), i(2, 3), workspace=small)):
        with pytest.raises(ds.DSparkError) as e:
            call()
        assert e.value.status == 1
