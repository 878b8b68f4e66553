"""GPU parity: truncated sampling, bit for bit against the integer oracle on the device's own
weights (expf's), and those weights against a 64-bit exponential."""
import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu


def _weights(x, T):
    """fl32 exp of fl32((x - m) * fl32(1 / T)) of each row on the device: the definition's weights."""
    import torch
    ok = torch.isfinite(x)
    m = torch.where(ok, x, -math.inf).amax(dim=1, keepdim=True)
    inv = (1.0 / torch.where(T == 0, torch.ones_like(T), T))[:, None].clamp(max=3.4028234663852886e38)
    w = torch.exp((x - m) * inv)
    w = torch.where(T[:, None] == 0, (x == m).float(), w)
    return torch.where(ok, w, torch.zeros_like(w))


class Rows:
    def __init__(self, logits, T, k, p, mp, u):
        import torch
        dev = lambda a, t: torch.tensor(np.asarray(a), dtype=t, device="cuda")
        self.logits = logits
        self.T, self.k, self.p = dev(T, torch.float32), dev(k, torch.int32), dev(p, torch.float32)
        self.mp, self.u = dev(mp, torch.float32), dev(u, torch.float32)

    def run(self, ds, probs=True, workspace=None):
        import torch
        out = torch.full(self.logits.shape, 9.0, device="cuda") if probs else None
        tok = ds.dspark_sample(self.logits, self.T, self.k, self.p, self.mp, self.u, probs=out, workspace=workspace)
        return tok, out

    def check(self, ds):
        x32 = self.logits.float()
        w = _weights(x32, self.T).cpu().numpy()
        tok, probs = self.run(ds)
        only, _ = self.run(ds, probs=False)
        tok, only, probs, x = tok.cpu().numpy(), only.cpu().numpy(), probs.cpu().numpy(), x32.cpu().numpy()
        par = [t.cpu().numpy() for t in (self.T, self.k, self.p, self.mp, self.u)]
        for r in range(len(tok)):
            token, kept, mass, total = oracle.sample_row(x[r], w[r], *(a[r] for a in par))
            assert tok[r] == token and only[r] == token, f"row {r}: token {tok[r]} ({only[r]}), oracle {token}"
            want = np.zeros(x.shape[1])
            for v, q in zip(kept, mass):
                want[v] = float(w[r][v]) * oracle.sample.MASS / total if q > 0 else 0.0
            np.testing.assert_array_equal(probs[r] > 0, want > 0, err_msg=f"row {r}: kept set")
            np.testing.assert_allclose(probs[r], want, rtol=2.0 ** -21)     # the total's rounding and a division
        return tok, probs


def _settings(rng, R):
    return (rng.choice([0.0, 0.3, 0.7, 1.0, 1.7], R), rng.choice([0, 1, 2, 17, 200, 10 ** 6], R),
            rng.choice([0.0, 0.1, 0.5, 0.9, 0.99, 1.0], R), rng.choice([0.0, 0.0, 0.01, 0.3, 1.0], R),
            rng.random(R).astype(np.float32))


def _normal(R, V, seed, gain=3.0, dtype=None):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, V, generator=g, device="cuda") * gain
    return x if dtype is None else x.to(dtype)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 1000, 4096, 5001, 50001])
def test_settings_and_vocabularies(cuda_lib, V, bf16):
    import torch
    R = 40 if V < 10000 else 12
    rng = np.random.default_rng(V)
    Rows(_normal(R, V, V, dtype=torch.bfloat16 if bf16 else None), *_settings(rng, R)).check(cuda_lib)


@pytest.mark.parametrize("R", [1, 2, 5, 17, 39, 77, 160, 400])
def test_row_counts(cuda_lib, R):
    rng = np.random.default_rng(R)
    Rows(_normal(R, 1500, R), *_settings(rng, R)).check(cuda_lib)


@pytest.mark.parametrize("bf16", [False, True])
def test_more_long_rows_than_blocks(cuda_lib, bf16):
    import torch
    R, V = 170, 40001
    rng = np.random.default_rng(V)
    Rows(_normal(R, V, V, dtype=torch.bfloat16 if bf16 else None), *_settings(rng, R)).check(cuda_lib)


@pytest.mark.parametrize("V,R", [(151936, 3), (151936, 41), (300007, 2), (1 << 21, 1)])
def test_large_vocabularies(cuda_lib, V, R):
    rng = np.random.default_rng(V + R)
    case = Rows(_normal(R, V, R), *_settings(rng, R))
    if R > 4:
        keep = slice(0, 3)
        tok, _ = case.run(cuda_lib)
        head = Rows(case.logits[keep].contiguous(), *(t[keep].cpu().numpy() for t in (case.T, case.k, case.p, case.mp,
                                                                                      case.u)))
        got, _ = head.check(cuda_lib)
        np.testing.assert_array_equal(tok[keep].cpu().numpy(), got)        # how rows are spread changes nothing
    else:
        case.check(cuda_lib)


def test_ties_flat_rows_and_few_values(cuda_lib):
    import torch
    rng = np.random.default_rng(1)
    V, R = 3000, 48
    x = torch.from_numpy(rng.integers(0, 4, (R, V)).astype(np.float32)).cuda()
    x[::3] = 2.5                                                          # every entry equal
    x[1::3, ::2] *= -0.0                                                  # zeros of both signs
    Rows(x, *_settings(rng, R)).check(cuda_lib)


def test_extreme_values_and_temperatures(cuda_lib):
    import torch
    rng = np.random.default_rng(2)
    R, V = 30, 700
    x = _normal(R, V, 3)
    x[0] *= 1e37
    x[1] *= 1e-39
    x[2, 5] = 3e38
    x[2, 6] = -3e38
    x[3:6, 10:600] = -math.inf
    x[6, 1:] = -math.inf
    x[7] = -3.4e38
    T = rng.choice([0.05, 1.0, 30.0], R).astype(np.float32)
    T[8], T[9], T[10], T[11] = 1e-38, 1e-42, 3e38, 1e-3
    _, k, p, mp, u = _settings(rng, R)
    u[12:14] = 0.0, np.float32(1) - np.float32(2.0 ** -24)
    Rows(x, T, k, p, mp, u).check(cuda_lib)


def test_nan_infinities_and_bad_settings_are_flagged(cuda_lib):
    ds = cuda_lib
    x = _normal(12, 500, 4)
    x[0, 3], x[1, 7], x[2] = math.nan, math.inf, -math.inf
    T, k, p, mp = np.ones(12, np.float32), np.zeros(12, int), np.full(12, 0.9), np.zeros(12)
    u = np.full(12, 0.4, np.float32)
    ws = ds.Workspace(ds.OP_SAMPLE, 12, 1, 500)
    tok, probs = Rows(x, T, k, p, mp, u).check(ds)
    assert tok[2] == 0 and not probs[2].any() and probs[0, 3] == 0 and probs[1, 7] == 0
    Rows(x, T, k, p, mp, u).run(ds, workspace=ws)
    assert ds.dspark_read_status(ws)[1] == ds.STATUS_NUMERIC
    x = _normal(12, 500, 5)
    clean = Rows(x, T, k, p, mp, u)
    clean.run(ds, workspace=ws)
    assert ds.dspark_read_status(ws) == (0, 0)
    bad = [("T", 0, math.nan, 0.0), ("T", 1, -1.0, 0.0), ("T", 2, math.inf, 0.0), ("p", 3, 1.5, 1.0), ("p", 4, -0.5, 0.0),
           ("p", 5, math.nan, 1.0), ("mp", 6, 2.0, 1.0), ("mp", 7, -1.0, 0.0), ("mp", 8, math.nan, 0.0),
           ("u", 9, 1.0, 1 - 2.0 ** -24), ("u", 10, -0.1, 0.0), ("u", 11, math.nan, 0.0)]
    for name, row, value, read_as in bad:
        one, same = Rows(x, T, k, p, mp, u), Rows(x, T, k, p, mp, u)
        getattr(one, name)[row] = value
        getattr(same, name)[row] = read_as
        a, pa = one.run(ds, workspace=ws)
        assert ds.dspark_read_status(ws)[1] == (ds.STATUS_NUMERIC if name == "T" else ds.STATUS_INPUT_RANGE)
        b, pb = same.run(ds)
        assert a.equal(b) and pa.equal(pb), (name, value)


def test_weights_are_the_exponential(cuda_lib):
    """probs of an untruncated row against a 64-bit softmax: the weights' 2 ulp of expf and three
    roundings ahead of it (difference, reciprocal, product: 1.5 ulp of the exponent, up to 28 of them)."""
    x = _normal(4, 20000, 6)
    T = np.array([0.5, 0.9, 1.0, 1.3], np.float32)
    _, probs = Rows(x, T, np.zeros(4, int), np.ones(4), np.zeros(4), np.full(4, 0.5)).run(cuda_lib)
    z = x.double().cpu().numpy() / T[:, None].astype(np.float64)
    p = np.exp(z - z.max(axis=1, keepdims=True))
    floor = 2.0 ** -40
    p = np.where(p >= floor * 1.01, p, 0) / p.sum(axis=1, keepdims=True)
    got = probs.cpu().numpy()
    big = p > 0
    np.testing.assert_allclose(got[big], p[big], rtol=28 * 1.5 * 2.0 ** -24 + 2.0 ** -20)


def test_streams_graphs_and_repeats(cuda_lib):
    import torch
    rng = np.random.default_rng(7)
    case = Rows(_normal(20, 30000, 8), *_settings(rng, 20))
    ws = cuda_lib.Workspace(cuda_lib.OP_SAMPLE, 20, 1, 30000)
    ws.buf.fill_(255)
    a, pa = case.run(cuda_lib, workspace=ws)
    tok, probs = torch.empty_like(a), torch.empty_like(pa)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cuda_lib.dspark_sample(case.logits, case.T, case.k, case.p, case.mp, case.u, tokens=tok, probs=probs,
                               workspace=ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, tok) and torch.equal(pa, probs)


def test_the_distribution_feeds_verification(cuda_lib):
    """Truncated target and draft rows verified without loss: the emitted first tokens follow the target."""
    import torch
    ds = cuda_lib
    B, V = 20000, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randn(1, V, generator=g, device="cuda") * 1.5
    d = t + torch.randn(1, V, generator=g, device="cuda")
    one = lambda v, ty=torch.float32: torch.full((B,), v, dtype=ty, device="cuda")
    u = torch.rand(B, generator=g, device="cuda")
    pt, pd = torch.empty(B, V, device="cuda"), torch.empty(B, V, device="cuda")
    ds.dspark_sample(t.expand(B, V).contiguous(), one(0.9), one(6, torch.int32), one(0.95), one(0.0), u, probs=pt)
    x = ds.dspark_sample(d.expand(B, V).contiguous(), one(0.9), one(5, torch.int32), one(0.9), one(0.0), u, probs=pd)
    out, _ = ds.dspark_verify(torch.stack([pt, pt], 1).contiguous(), pd[:, None].contiguous(), x[:, None].contiguous(),
                              None, 11, 0)
    got = np.bincount(out[:, 0].cpu().numpy(), minlength=V)
    want = pt[0].cpu().numpy().astype(np.float64)
    assert got[want == 0].sum() == 0
    keep = want > 0
    chi2 = ((got[keep] - B * want[keep]) ** 2 / (B * want[keep])).sum()
    assert chi2 < 30.0                                                     # 5 degrees of freedom: p < 2e-5


def test_refusals(cuda_lib):
    import torch
    ds = cuda_lib
    c = Rows(_normal(3, 100, 9), np.ones(3), np.zeros(3, int), np.ones(3), np.zeros(3), np.full(3, 0.5))
    with pytest.raises(TypeError):
        ds.dspark_sample(c.logits.half(), c.T, c.k, c.p, c.mp, c.u)
    with pytest.raises(TypeError):
        ds.dspark_sample(c.logits, c.T, c.k.long(), c.p, c.mp, c.u)
    with pytest.raises(ValueError):
        ds.dspark_sample(c.logits, c.T[:2], c.k, c.p, c.mp, c.u)
    with pytest.raises(ValueError):
        ds.dspark_sample(c.logits, c.T, c.k, c.p, c.mp, c.u, probs=torch.empty(3, 99, device="cuda"))
    with pytest.raises(ds.DSparkError) as e:
        ds.dspark_sample(torch.zeros(1, (1 << 21) + 1, device="cuda"), c.T[:1], c.k[:1], c.p[:1], c.mp[:1], c.u[:1])
    assert e.value.status == 1
