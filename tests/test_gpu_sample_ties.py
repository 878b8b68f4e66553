"""GPU parity: top-p whose boundary lies between large groups of equal logits, against the integer
definition on the device's own weights.

The kernels narrow the range that holds the cut by bounds of the masses; where two groups of equal
logits meet at the wanted mass, bounds cannot part them and exact sums have to.
"""
import numpy as np
import pytest

import oracle
from tests.test_gpu_sample import Rows, _settings, _weights

pytestmark = pytest.mark.gpu
MASS, FRAC = 1 << 40, 1 << 24


def definition(x, w, T, k, p, mp, u):
    """oracle.sample_row with sorted arrays instead of loops: (token, kept ids, their masses, total)."""
    ids = np.argsort(-x, kind="stable")                                  # equal ones by id
    ids = ids[np.isfinite(x[ids])]
    k = 1 if T == 0 else (int(k) if k > 0 else len(x))
    ids = ids[:k]
    ids = ids[w[ids] >= np.float32(mp)]
    mass = np.floor(w[ids].astype(np.float64) * MASS).astype(np.int64)   # exact; sums stay below 2^62
    need = int(mass.sum()) * int(np.floor(float(p) * FRAC)) // FRAC
    kept = mass.cumsum() - mass < need
    kept[0] = True
    ids, mass = ids[kept], mass[kept]
    total = int(mass.sum())
    target = total * int(np.floor(float(u) * FRAC)) // FRAC
    by_id = np.argsort(ids)
    return int(ids[by_id][np.searchsorted(mass[by_id].cumsum(), target, side="right")]), ids, mass, total


def check(ds, case, oracle_rows=2):
    x = case.logits.float()
    w = _weights(x, case.T).cpu().numpy()
    tok, probs = case.run(ds)
    only, _ = case.run(ds, probs=False)
    tok, only, probs, x = tok.cpu().numpy(), only.cpu().numpy(), probs.cpu().numpy(), x.cpu().numpy()
    par = [t.cpu().numpy() for t in (case.T, case.k, case.p, case.mp, case.u)]
    for r in range(len(tok)):
        token, kept, mass, total = definition(x[r], w[r], *(a[r] for a in par))
        if r < oracle_rows:
            t2, k2, m2, q2 = oracle.sample_row(x[r], w[r], *(a[r] for a in par))
            assert (t2, k2, m2, q2) == (token, kept.tolist(), mass.tolist(), total)
        want = np.zeros(x.shape[1])
        want[kept] = np.where(mass > 0, w[r][kept].astype(np.float64) * MASS / total, 0.0)
        assert (probs[r] > 0).sum() == (want > 0).sum(), f"row {r}: {(probs[r] > 0).sum()} kept for {(want > 0).sum()}"
        np.testing.assert_array_equal(probs[r] > 0, want > 0, err_msg=f"row {r}: kept set")
        np.testing.assert_allclose(probs[r], want, rtol=2.0 ** -21)      # the total's rounding and a division
        assert tok[r] == token and only[r] == token, f"row {r}: token {tok[r]} ({only[r]}) for {token}"


def rows_of(groups, V, seed, bf16=False, more=()):
    """One row per boundary and step: the groups (count, logit) shuffled, entries between them or below for
    the rest of the row, and top-p set on each boundary between groups, to 3 units of 2^-24 either side."""
    import torch
    rng = np.random.default_rng(seed)
    x = np.concatenate([np.full(n, v, np.float32) for n, v in groups] + [np.asarray(more, np.float32)])
    x = np.concatenate([x, np.full(V - len(x), -40.0, np.float32)])      # mass 0
    x = x[rng.permutation(V)]
    t = torch.from_numpy(x).cuda()
    if bf16:
        t = t.to(torch.bfloat16)
    w = _weights(t.float()[None], torch.ones(1, device="cuda"))[0].cpu().numpy().astype(np.float64)
    values = t.float().cpu().numpy()
    mass = np.floor(w * MASS)
    P = []
    for _, v in groups:
        edge = mass[values >= np.float32(torch.tensor(v).to(t.dtype).float().item())].sum() / mass.sum() * FRAC
        P += [min(FRAC, int(edge) + d) for d in range(-3, 5)]
    R = len(P)
    return Rows(t.repeat(R, 1), np.ones(R), np.zeros(R, int), np.array(P) / FRAC, np.zeros(R), rng.random(R).astype(np.float32))


def repeated(case, R):
    """The case's rows again and again, R of them."""
    import torch
    at = torch.arange(R, device="cuda") % case.logits.shape[0]
    for name in ("logits", "T", "k", "p", "mp", "u"):
        setattr(case, name, getattr(case, name)[at].contiguous())
    return case


GROUPS = {
    "near": [(3000, 0.0), (3000, -1e-5)],
    "half": [(2500, 0.0), (3500, -0.5)],
    "three": [(2100, 1.0), (2500, 0.25), (2900, -1.0)],
    "small_first": [(1, 3.0), (2600, 0.5), (2600, 0.0)],
    "wide": [(2200, 5.0), (5000, -20.0)],
}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_top_p_on_the_boundary_of_tied_groups_one_block(cuda_lib, name, bf16):
    check(cuda_lib, rows_of(GROUPS[name], 8000, 1, bf16))


@pytest.mark.parametrize("name", sorted(GROUPS))
def test_top_p_on_the_boundary_of_tied_groups_clusters(cuda_lib, name):
    case = rows_of([(3 * n, v) for n, v in GROUPS[name]], 24001, 2)
    check(cuda_lib, repeated(case, 9))
    check(cuda_lib, repeated(rows_of([(3 * n, v) for n, v in GROUPS[name]], 24001, 3), 40))


@pytest.mark.parametrize("name", sorted(GROUPS))
def test_top_p_on_the_boundary_of_tied_groups_queue(cuda_lib, name):
    check(cuda_lib, repeated(rows_of(GROUPS[name], 8003, 4), 170))
    check(cuda_lib, repeated(rows_of([(9 * n, v) for n, v in GROUPS[name]], 70001, 5), 160))


def test_the_stated_rows(cuda_lib):
    import torch
    x = torch.zeros(2, 6000, device="cuda")
    x[0, 3000:] = -1e-5
    x[1, 2500:] = -0.5
    case = Rows(x, np.ones(2), np.zeros(2, int), [0.5, 0.54076], np.zeros(2), [0.3, 0.999])
    _, probs = case.run(cuda_lib)
    assert (probs > 0).sum(dim=1).tolist() == [3000, 2500]
    check(cuda_lib, case)


def test_sparse_entries_between_groups(cuda_lib):
    """Few entries between the groups: a range that loses some of them at each level and keeps the groups."""
    rng = np.random.default_rng(6)
    for scale in (1.0, 1e-3, 1e-6):
        more = np.concatenate([-rng.random(300), -rng.random(100) * 1e-2, -1 + rng.random(100) * 1e-2]) * scale
        check(cuda_lib, rows_of([(2500, 0.0), (2500, -scale)], 7900, 7, more=more))
        check(cuda_lib, rows_of([(5500, 0.0), (5500, -scale)], 17900, 8, more=more))


def test_with_top_k_and_min_p(cuda_lib):
    for top_k, min_p in ((4000, 0.0), (5200, 0.0), (0, 0.5), (0, 0.999), (5300, 0.5)):
        for V, seed in ((8000, 9), (24001, 10)):
            case = rows_of([(2500, 0.0), (2700, -0.5), (2800, -0.75)], V, seed)
            case.k[:], case.mp[:] = top_k, min_p
            x, w = case.logits.float().cpu().numpy(), _weights(case.logits, case.T).cpu().numpy()
            P = []                                                       # the boundaries of what those leave
            for r in range(len(x)):
                _, ids, mass, total = definition(x[r], w[r], 1.0, top_k, 1.0, min_p, 0.0)
                edge = mass[x[r][ids] >= (0.0, -0.5)[r % 2]].sum() / total * FRAC
                P.append(min(FRAC, int(edge) + r // 2 % 8 - 3) / FRAC)
            case.p[:] = case.p.new_tensor(P)
            check(cuda_lib, case)


@pytest.mark.parametrize("V,R", [(8000, 60), (32000, 12), (32000, 400)])
def test_integer_logits(cuda_lib, V, R):
    import torch
    g = torch.Generator(device="cuda").manual_seed(V + R)
    x = (torch.randn(R, V, generator=g, device="cuda") * 3).round()
    rng = np.random.default_rng(R)
    T, k, _, mp, u = _settings(rng, R)
    k[R // 2:], mp[R // 2:], T[R // 2:] = 0, 0.0, 1.0
    case = Rows(x, T, k, rng.random(R).astype(np.float32), mp, u)
    w, x = _weights(x, case.T).cpu().numpy(), x.cpu().numpy()
    for r in range(R // 2, R):                                           # every one of these on a boundary
        _, ids, mass, total = definition(x[r], w[r], 1.0, 0, 1.0, 0.0, 0.0)
        edge = mass[x[r][ids] >= rng.integers(-4, 5)].sum() / total * FRAC
        case.p[r] = min(FRAC, int(edge) + int(rng.integers(-1, 3))) / FRAC
    check(cuda_lib, case)
