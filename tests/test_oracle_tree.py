"""Pins of the tree operators' oracles: chains against the chain's own oracles, hand-worked trees, laws."""
import numpy as np
import pytest

import oracle
from tests._trees import random_parents


def test_a_chain_is_a_causal_window():
    for L, n in ((9, 4), (4, 4), (1, 1)):
        for i in range(n):
            parents = list(range(-1, n - 1))
            assert oracle.tree_row_sees(L, n, i, parents) == list(range(L - n + i + 1))
            for window, sinks in ((n, 0), (n + 1, 2), (100, 3)):
                assert oracle.tree_row_sees(L, n, i, parents, window, sinks) == oracle.window_row_sees(L, n, i, window, sinks)


def test_windows_worked_by_hand():
    assert oracle.window_row_sees(10, 2, 0, 3, 0) == [6, 7, 8]
    assert oracle.window_row_sees(10, 2, 1, 3, 2) == [0, 1, 7, 8, 9]
    assert oracle.window_row_sees(10, 2, 0, 3, 2, causal=False) == [0, 1, 6, 7, 8, 9]
    assert oracle.window_row_sees(2, 4, 0, 3, 0) == [] and oracle.window_row_sees(2, 4, 2, 1, 0) == [0]


def test_a_tree_worked_by_hand():
    #     0 - 1 - 3
    #      \   \- 4 - 5        2: a second child of the root
    parents = [-1, 0, 0, 1, 1, 4]
    assert oracle.depths(parents) == [0, 1, 1, 2, 2, 3]
    assert oracle.tree_row_sees(8, 6, 5, parents) == [0, 1, 2, 3, 6, 7]
    assert oracle.tree_row_sees(8, 6, 2, parents) == [0, 1, 2, 4]
    assert oracle.tree_row_sees(28, 6, 5, parents, 6, 1) == [0, 20, 21, 22, 23, 26, 27]      # position 25
    tokens = [9, 5, 6, 7, 7, 8]
    target = {0: 5, 1: 7, 3: 2, 4: 8, 5: 1, 2: 0}
    # two children of node 1 hold 7: the first counts, and its target has no child
    assert oracle.verify_tree(target.get, parents, tokens, 6) == ([5, 7, 2], [0, 1, 3])
    assert oracle.verify_tree({**target, 0: 6}.get, parents, tokens, 6) == ([6, 0], [0, 2])
    assert oracle.verify_tree(target.get, parents, tokens, 3) == ([5, 7], [0, 1])            # the nodes behind do not exist
    assert oracle.verify_tree(target.get, parents, tokens, 0) == ([], [])


def test_a_greedy_chain_is_greedy_verification():
    rng = np.random.default_rng(0)
    for _ in range(50):
        gamma, V = int(rng.integers(1, 6)), 3
        target = rng.standard_normal((1, gamma + 1, V)).astype(np.float32)
        draft = rng.integers(0, V, (1, gamma))
        want, accepted = oracle.verify_greedy(target, draft)[:2]
        out, path = oracle.verify_tree(lambda k: int(target[0, k].argmax()), list(range(-1, gamma)), [0] + draft[0].tolist(), gamma + 1)
        assert len(path) - 1 == int(accepted[0]) and out == [int(t) for t in want[0] if t >= 0]


def test_a_sampled_tree_keeps_the_target_law():
    """The first two tokens put out have the target's joint law, whatever the tree proposes (chi-squared, 8 cells)."""
    from scipy.stats import chi2
    rng = np.random.default_rng(1)
    V, trials = 3, 20000
    first = np.array([0.5, 0.3, 0.2])
    second = np.array([[0.2, 0.2, 0.6], [0.7, 0.1, 0.2], [0.1, 0.8, 0.1]])
    parents, tokens = [-1, 0, 0, 1], [0, 0, 2, 2]           # the tree proposes 0 or 2, and 2 behind 0
    count = np.zeros((V, V))
    for _ in range(trials):
        u = rng.random(8)

        def next_token(node):
            p = first if node == 0 else second[tokens[node]] if parents[node] == 0 else np.full(V, 1 / V)
            return int(np.searchsorted(np.cumsum(p), u[node], side="right").clip(max=V - 1))

        out, _ = oracle.verify_tree(next_token, parents, tokens, 4)
        a = out[0]
        b = out[1] if len(out) > 1 else int(np.searchsorted(np.cumsum(second[a]), u[7], side="right").clip(max=V - 1))
        count[a, b] += 1
    want = first[:, None] * second * trials
    assert ((count - want) ** 2 / want).sum() < chi2.ppf(1 - 1e-6, V * V - 1)


def test_random_parents_come_before_their_nodes():
    rng = np.random.default_rng(2)
    for shape in ("random", "chain", "star", "forest"):
        p = random_parents(rng, 4, 20, deepest=5, shape=shape)
        assert (p < np.arange(20)).all() and (p[:, 0] == -1).all()
    assert max(oracle.depths(random_parents(rng, 1, 60, deepest=3)[0])) <= 3


def test_compact_and_copy_touch_nothing_else():
    rng = np.random.default_rng(3)
    cache = rng.standard_normal((2, 5, 3, 4, 8))
    table = [3, 0, 4]
    new, length = oracle.compact(cache, table, 11, 6, [0, 2, 5], 2)
    assert length == 8
    flat = lambda c, j: c[:, table[j // 4], :, j % 4]
    np.testing.assert_array_equal(flat(new, 5), flat(cache, 5))
    np.testing.assert_array_equal(flat(new, 6), flat(cache, 7))
    np.testing.assert_array_equal(flat(new, 7), flat(cache, 10))
    for j in (0, 1, 2, 3, 4, 8, 9, 10, 11):
        np.testing.assert_array_equal(flat(new, j), flat(cache, j))
    np.testing.assert_array_equal(new[:, [1, 2]], cache[:, [1, 2]])
    copied = oracle.copy_pages(cache, [1, 1], [2, 0], [4, 1])
    np.testing.assert_array_equal(copied[:, 2], cache[:, 1])
    np.testing.assert_array_equal(copied[:, 0, :, :1], cache[:, 1, :, :1])
    np.testing.assert_array_equal(copied[:, 0, :, 1:], cache[:, 0, :, 1:])
    with pytest.raises(IndexError):
        oracle.copy_pages(cache, [9], [0])
