"""The tree oracle against closed forms, other formulations and brute force
(CPU only)."""
import itertools
import math

import numpy as np
import pytest

import oracle


def test_visibility_forms_agree():
    parents = [-1, 0, 0, 1, 1, 2, 5]
    sees = oracle.visible_nodes(7, parents=parents)
    assert [sorted(np.flatnonzero(r)) for r in sees] == \
        [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 4], [0, 2, 5], [0, 2, 5, 6]]
    mask = [sum(1 << int(j) for j in np.flatnonzero(r)) for r in sees]
    assert (oracle.visible_nodes(7, mask=mask) == sees).all()
    chain = [-1, 0, 1, 2, 3, 4, 5]
    assert (oracle.visible_nodes(7, parents=chain) == oracle.visible_nodes(7)).all()


def _tiny(rng, B=2, H=2, G=2, D=4, page=4, T=3):
    N = B * T
    pool = 9
    k, v = rng.standard_normal((2, pool, H, page, D))
    table = rng.permutation(pool)[: B * 4].reshape(B, 4)
    q = rng.standard_normal((N, H * G, D))
    kn, vn = rng.standard_normal((2, N, H, D))
    return q, kn, vn, k, v, table, np.arange(B + 1) * T


def test_attention_of_equal_keys_is_the_mean_of_the_values():
    rng = np.random.default_rng(1)
    q, kn, vn, k, v, table, off = _tiny(rng)
    k[:] = 0.5
    kn[:] = 0.5
    lens = [5, 0]
    out, lse, _ = oracle.tree_attention_ref(q, kn, vn, k, v, table, lens, off, 0.7)
    flat = np.concatenate([v[p, 1] for p in table[0]])[:5]
    want = np.concatenate([flat, vn[:2, 1]]).mean(0)
    np.testing.assert_allclose(out[1, 2], want, atol=1e-12)
    assert lse[1, 2] == pytest.approx(0.35 * q[1, 2].sum() + math.log(7))
    np.testing.assert_allclose(out[3, 0], vn[3, 0], atol=1e-12)      # a root alone sees itself


def test_attention_does_not_depend_on_where_the_split_into_cache_and_tree_is():
    """A chain of three nodes equals the last node over a cache that holds
    the first two."""
    rng = np.random.default_rng(2)
    q, kn, vn, k, v, table, off = _tiny(rng, B=1)
    a, la, _ = oracle.tree_attention_ref(q, kn, vn, k, v, table, [6], off, 0.5)
    for i in range(2):
        t = 6 + i
        k[table[0, t // 4], :, t % 4], v[table[0, t // 4], :, t % 4] = kn[i], vn[i]
    b, lb, _ = oracle.tree_attention_ref(q[2:], kn[2:], vn[2:], k, v, table, [8], np.array([0, 1]), 0.5)
    np.testing.assert_allclose(a[2], b[0], atol=1e-12)
    np.testing.assert_allclose(la[2], lb[0], atol=1e-12)


def test_weights_of_a_branch_sum_to_its_rows():
    """Each row's attention weights sum to one, so a branch of m rows and G
    heads gives m * G in all."""
    rng = np.random.default_rng(3)
    q, kn, vn, k, v, table, off = _tiny(rng, B=1)
    lens = [7]
    _, lse, _ = oracle.tree_attention_ref(q, kn, vn, k, v, table, lens, off, 0.5)
    w = oracle.commit_weights_ref(q[:, 2:4], lse[:, 2:4], kn, k, table[0], 7, [0, 1, 2], 1, 0.5)
    assert w.sum() == pytest.approx(6.0)


def test_rows_that_saw_nothing_give_no_weight():
    rng = np.random.default_rng(7)
    q, kn, vn, k, v, table, off = _tiny(rng, B=1)
    _, lse, _ = oracle.tree_attention_ref(q, kn, vn, k, v, table, [0], off, 0.5, mask=[0, 2, 6])
    assert lse[0, 2] == -math.inf and np.isfinite(lse[1:]).all()
    w = oracle.commit_weights_ref(q[:, 2:4], lse[:, 2:4], kn, k, table[0], 0, [0, 1], 1, 0.5)
    one = oracle.commit_weights_ref(q[1:, 2:4], lse[1:, 2:4], kn[1:], k, table[0], 0, [0], 1, 0.5)
    assert w[1] == pytest.approx(one[0]) == pytest.approx(2.0)


def test_greedy_walk_against_all_branches():
    """The walk's branch is the longest one whose every token is its parent's
    argmax, the lowest sibling first."""
    rng = np.random.default_rng(4)
    for _ in range(200):
        T, V = int(rng.integers(1, 9)), 4
        parents = np.array([-1] + [int(rng.integers(0, i)) for i in range(1, T)])
        logits, tokens = rng.standard_normal((T, V)), rng.integers(0, V, T)
        acc, path, out = oracle.tree_verify_greedy_ref(logits, tokens, parents, [0, T], 8)
        best = logits.argmax(1)
        ok = [True] * T
        for c in range(1, T):
            sib = [s for s in range(1, c) if parents[s] == parents[c] and tokens[s] == tokens[c]]
            ok[c] = ok[parents[c]] and tokens[c] == best[parents[c]] and not sib
        want = [c for c in range(T) if ok[c]]
        assert list(path[0][: acc[0] + 1]) == want and acc[0] == len(want) - 1
        assert list(out[0][: acc[0] + 1]) == [best[c] for c in want]
        assert (path[0][acc[0] + 1:] == -1).all() and (out[0][acc[0] + 1:] == -1).all()


def test_walk_without_bonus_stops_at_a_leaf():
    logits = np.eye(3)
    acc, path, out = oracle.tree_verify_greedy_ref(logits, [9, 0, 1], [-1, 0, 1], [0, 3], 3, no_bonus=True)
    assert acc[0] == 2 and list(path[0]) == [0, 1, 2] and list(out[0]) == [0, 1, -1]


def test_eviction_keeps_the_best_subset():
    rng = np.random.default_rng(5)
    for _ in range(100):
        n, budget = int(rng.integers(1, 8)), int(rng.integers(1, 8))
        mass = rng.permutation(n).astype(float)
        src = oracle.evict_ref(mass, None, n, 0, budget, 0, 0)
        assert len(src) == min(n, budget) == len(set(src))
        best = max(itertools.combinations(range(n), min(n, budget)), key=lambda s: mass[list(s)].sum())
        assert set(src) == set(best)
        assert all(s == i for i, s in enumerate(src) if i in best)       # those below the budget stay
        moved = [s for i, s in enumerate(src) if i not in best]
        assert moved == sorted(moved) and all(s >= budget for s in moved)


def test_eviction_protects_positions():
    pos = np.array([3, 0, 1, 2, 4, 5])
    src = oracle.evict_ref(np.array([9.0, 0, 8, 7, 0, 0]), pos, 6, 6, 3, 2, 1)
    assert set(src) == {1, 4, 5}
    assert src == [4, 1, 5]


def test_eviction_protects_what_is_at_or_past_seen_also_without_a_recent_window():
    """Tokens just appended, before `seen` counts them."""
    pos = np.array([0, 1, 2, 3, 10, 11])
    assert oracle.evict_ref(np.array([9.0, 8, 7, 6, 0, 0]), pos, 6, 10, 3, 0, 0) == [0, 4, 5]
    assert oracle.evict_ref(np.array([9.0, 8, 7, 6, 0, 0]), pos, 6, 12, 3, 0, 0) == [0, 1, 2]


def test_beam_against_a_full_sort():
    rng = np.random.default_rng(6)
    z, s = rng.standard_normal((3, 11)), rng.standard_normal(3)
    p = z - np.log(np.exp(z).sum(1, keepdims=True)) + s[:, None]
    got = oracle.beam_select_ref(z, s, 7)
    order = np.argsort(-p.ravel(), kind="stable")[:7]
    assert [(w, v) for _, w, v in got] == [(i // 11, i % 11) for i in order]
    np.testing.assert_allclose([x for x, _, _ in got], p.ravel()[order])
    ended = oracle.beam_select_ref(z, np.array([0.0, 5.0, -np.inf]), 3, ended=[0, 1, 0], eos=4)
    assert ended[0] == (5.0, 1, 4) and all(w == 0 for _, w, _ in ended[1:])


def test_beam_scores_do_not_depend_on_the_level_of_the_logits():
    z = np.array([[2.0, 1.0, 0.0, 2.0]])
    want = oracle.beam_select_ref(z, np.zeros(1), 4)
    for level in (-1e4, 2.0 ** 40):
        got = oracle.beam_select_ref(z + level, np.zeros(1), 4)
        assert [c[1:] for c in got] == [c[1:] for c in want]
        np.testing.assert_allclose([c[0] for c in got], [c[0] for c in want], atol=1e-12)
    flat = oracle.beam_select_ref(np.full((1, 8), -3e38), np.zeros(1), 2)
    assert [c[1:] for c in flat] == [(0, 0), (0, 1)] and flat[0][0] == pytest.approx(-math.log(8))
