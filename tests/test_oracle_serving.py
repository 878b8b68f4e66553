"""Pins of the serving operators' oracles: closed forms and brute force on tiny inputs."""
import itertools
import math

import numpy as np
import pytest

import oracle


def test_rotation_is_a_complex_product_and_keeps_relative_positions():
    rng = np.random.default_rng(0)
    D, rot = 16, 12
    freq = 10.0 ** -np.arange(rot // 2)
    x = rng.standard_normal((5, 3, D))
    pos = np.array([0, 1, 7, 30, 1000])
    ang = pos[:, None] * freq
    for interleaved in (False, True):
        y = oracle.rotate(x, np.cos(ang), np.sin(ang), interleaved)
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
        z = (a + 1j * b) * np.exp(1j * ang)[:, None]
        ya, yb = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        np.testing.assert_allclose(ya + 1j * yb, z, atol=1e-12)
        np.testing.assert_array_equal(y[..., rot:], x[..., rot:])
        np.testing.assert_array_equal(y[0], x[0])
    # the dot product of two rotated vectors depends on the distance of their positions only
    q, k = rng.standard_normal((1, 1, D)), rng.standard_normal((1, 1, D))

    def dot(p, r):
        turn = lambda v, t: oracle.rotate(v, np.cos(t * freq)[None], np.sin(t * freq)[None])
        return float((turn(q, p) * turn(k, r)).sum())

    assert dot(3, 10) == pytest.approx(dot(20, 27), abs=1e-10)


def test_rms_norm_closed_form():
    assert oracle.rms_norm(np.array([3.0, 4.0]), np.array([1.0, 2.0]), 0.0) == pytest.approx(
        np.array([3.0, 8.0]) / math.sqrt(12.5))


def test_append_writes_only_the_named_slots():
    rng = np.random.default_rng(1)
    K, V = rng.standard_normal((3, 2, 4, 16)), rng.standard_normal((3, 2, 4, 16))
    k, v = rng.standard_normal((3, 2, 16)), rng.standard_normal((3, 2, 16))
    cs = np.concatenate([np.ones((5, 8)), np.zeros((5, 8))], axis=1)       # angle 0 everywhere
    _, K2, V2 = oracle.kv_append(None, k, v, [0, 1, 4], [9, -1, 2], cs, K, V)
    np.testing.assert_array_equal(K2[2, :, 1], k[0])
    np.testing.assert_array_equal(V2[0, :, 2], v[2])
    K2[2, :, 1], K2[0, :, 2] = K[2, :, 1], K[0, :, 2]
    V2[2, :, 1], V2[0, :, 2] = V[2, :, 1], V[0, :, 2]
    np.testing.assert_array_equal(K2, K)
    np.testing.assert_array_equal(V2, V)


def test_attention_closed_forms():
    # equal keys: the mean of the values; one huge score: that value; no key: zero
    V = np.arange(12.0).reshape(4, 3)
    out, lse, _, _ = oracle.attend_row(np.ones(3), np.ones((4, 3)), V, 0.5)
    np.testing.assert_allclose(out, V.mean(axis=0))
    assert lse == pytest.approx(1.5 + math.log(4))
    K = np.zeros((4, 3))
    K[2, 0] = 1e4
    np.testing.assert_allclose(oracle.attend_row(np.array([1.0, 0, 0]), K, V, 1.0)[0], V[2])
    out, lse, _, _ = oracle.attend_row(np.ones(3), np.zeros((0, 3)), np.zeros((0, 3)), 1.0)
    assert not out.any() and lse == -math.inf


def test_paged_equals_prompt_on_the_same_tokens():
    """The last n rows of a prompt are a window over the cache that holds it, whatever the pages' order."""
    rng = np.random.default_rng(2)
    L, Hkv, G, D, page, n = 21, 2, 3, 8, 4, 5
    q, k, v = rng.standard_normal((L, Hkv * G, D)), rng.standard_normal((L, Hkv, D)), rng.standard_normal((L, Hkv, D))
    pages = rng.permutation(9)[:6]
    K, V = np.full((9, Hkv, page, D), np.nan), np.full((9, Hkv, page, D), np.nan)
    for j in range(L):
        K[pages[j // page], :, j % page], V[pages[j // page], :, j % page] = k[j], v[j]
    for causal in (True, False):
        a = oracle.prompt_attention(q, k, v, [0, L], 0.3, causal)
        b = oracle.paged_attention(q[None, -n:], K, V, pages[None], [L], 0.3, None, causal)
        np.testing.assert_allclose(b[0][0], a[0][-n:], atol=1e-12)
        np.testing.assert_allclose(b[1][0], a[1][-n:], atol=1e-12)


def test_packed_sequences_do_not_see_each_other():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 1, 4)), rng.standard_normal((9, 1, 4))
    whole = oracle.prompt_attention(q, k, v, [0, 4, 4, 9], 0.5)[0]
    for a, z in ((0, 4), (4, 9)):
        np.testing.assert_array_equal(whole[a:z], oracle.prompt_attention(q[a:z], k[a:z], v[a:z], [0, z - a], 0.5)[0])


def test_truncation_by_brute_force():
    """Every setting on a tiny vocabulary against the definition of each filter as a set."""
    rng = np.random.default_rng(4)
    x = np.round(rng.standard_normal(7), 1)
    x[5] = x[2]                                                            # a tie: the lower id comes first
    for T, k, p, mp in itertools.product((0.5, 1.0, 2.0), (0, 1, 3, 7), (0.0, 0.3, 0.8, 1.0), (0.0, 0.2, 1.0)):
        w = np.exp((x - x.max()) / T)
        order = sorted(range(7), key=lambda v: (-x[v], v))
        kept = [v for v in order[:k or 7] if w[v] >= np.float32(mp)]
        best = next(n for n in range(1, len(kept) + 1) if w[kept[:n]].sum() >= p * w[kept].sum() * (1 - 1e-7))
        want = np.zeros(7)
        want[kept[:best]] = w[kept[:best]] / w[kept[:best]].sum()
        np.testing.assert_allclose(oracle.truncated_distribution(x, T, k, p, mp), want, atol=1e-9)


def test_draw_follows_the_distribution():
    x = np.array([0.0, 1.0, -1.0, 2.0, -np.inf])
    w = oracle.weights(x, 1.0)
    n = 1 << 12
    got = np.bincount([oracle.sample_row(x, w, 1.0, 3, 1.0, 0.0, (i + 0.5) / n)[0] for i in range(n)], minlength=5) / n
    np.testing.assert_allclose(got, oracle.truncated_distribution(x, 1.0, 3, 1.0, 0.0), atol=1.5 / n)
    assert oracle.sample_row(x, oracle.weights(x, 0.0), 0.0, 0, 1.0, 0.0, 0.9)[0] == 3
    assert oracle.sample_row(np.full(3, -np.inf), np.zeros(3), 1.0, 0, 1.0, 0.0, 0.5)[0] == 0
