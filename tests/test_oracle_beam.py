"""Pins of the beam and eviction oracles (CPU): brute force over sequences, plain sums of probabilities, permutation invariance."""

import itertools

import numpy as np
import pytest

import oracle
from oracle import beam, evict


def _log_softmax(x):
    x = x - x.max(-1, keepdims=True)
    return x - np.log(np.exp(x).sum(-1, keepdims=True))


def test_a_wide_enough_search_finds_the_best_sequences():
    # logits depend on the last token alone; beams wide enough for every prefix make the search exhaustive
    V, K = 3, 9
    table = np.random.default_rng(0).standard_normal((V, V))
    tokens, scores = [[[0]]], np.array([[0.0]])
    for _ in range(2):
        W = scores.shape[1]
        r = beam.beam_select(np.array([[table[s[-1]] for s in tokens[0]]]), scores, min(K, W * V))
        tokens = [[tokens[0][p] + [int(t)] for p, t in zip(r["parent"][0], r["token"][0])]]
        scores = r["score"]
    lp = _log_softmax(table)
    best = sorted(((lp[0, a] + lp[a, b], [0, a, b]) for a, b in itertools.product(range(V), repeat=2)), reverse=True)
    assert tokens[0] == [s for _, s in best[:K]]
    np.testing.assert_allclose(scores[0], [v for v, _ in best[:K]], atol=1e-12)


def test_ended_dead_and_masked_beams():
    x = np.zeros((1, 4, 3))
    x[0, 0, 1] = -np.inf
    x[0, 0, 2] = np.nan
    x[0, 2] = [0.0, np.inf, 0.0]
    r = beam.beam_select(x, np.array([[-1.0, -2.0, 0.0, -np.inf]]), 4, eos=2, ended=np.array([[0, 1, 0, 0]]), length=np.array([[3, 7, 3, 3]]))
    assert r["token"].tolist() == [[0, 2, -1, -1]] and r["parent"].tolist() == [[0, 1, -1, -1]]
    assert r["ended"].tolist() == [[0, 1, 1, 1]] and r["length"].tolist() == [[4, 7, 0, 0]]
    assert r["score"].tolist() == [[-1.0, -2.0, -np.inf, -np.inf]]


def test_equal_pairs_go_to_the_lower_beam_and_token():
    r = beam.beam_select(np.zeros((1, 2, 4)), np.array([[-1.0, -1.0]]), 6)
    assert list(zip(r["parent"][0], r["token"][0])) == [(0, 0), (0, 1), (0, 2), (0, 3), (1, 0), (1, 1)]
    # weighed by length the longer of two beams of equal score is ahead
    r = beam.beam_select(np.zeros((1, 2, 4)), np.array([[-1.0, -1.0]]), 1, length=np.array([[1, 5]]), alpha=1.0)
    assert r["parent"][0, 0] == 1


def test_reorders():
    rng = np.random.default_rng(1)
    parent = np.array([[2, 0, 0], [1, -1, 5]])
    x = rng.standard_normal((2, 3, 4))
    y = beam.reorder(x, parent)
    np.testing.assert_array_equal(y[0], x[0, [2, 0, 0]])
    np.testing.assert_array_equal(y[1], x[1, [1, 1, 2]])
    cache = rng.standard_normal((6, 2, 5, 4))
    z = beam.kv_reorder(cache, parent, [1, 0], [4, 6])
    np.testing.assert_array_equal(z[0, :, 1:4], cache[2, :, 1:4])
    np.testing.assert_array_equal(z[:, :, [0, 4]], cache[:, :, [0, 4]])
    np.testing.assert_array_equal(z[3:], cache[3:])          # the range leaves the cache
    table = rng.permutation(18).reshape(6, 3)
    pool = rng.standard_normal((18, 2, 2, 4))
    flat = lambda p: p[table].transpose(0, 2, 1, 3, 4).reshape(6, 2, 6, 4)  # noqa: E731
    np.testing.assert_array_equal(flat(beam.kv_reorder(pool, parent, [1, 2], [4, 6], table)), beam.kv_reorder(flat(pool), parent, [1, 2], [4, 6]))


def test_weights_are_the_sums_of_the_attention_s_probabilities():
    # a chain's attention in one matrix: the columns' sums of its softmax
    rng = np.random.default_rng(2)
    n, r, D = 9, 4, 8
    q, k = rng.standard_normal((1, 2, r, D)), rng.standard_normal((1, 1, n, D))
    s = np.einsum("hid,jd->hij", q[0], k[0, 0]) / np.sqrt(D)
    s[:, np.arange(n)[None] > (n - r + np.arange(r))[:, None]] = -np.inf
    p = np.exp(_log_softmax(s))
    lse = np.log(np.exp(s).sum(-1))[None]
    acc = rng.standard_normal((1, 1, n + 2))
    new, pos, _ = evict.kv_weigh(q, lse, k, [n], acc, np.full((1, 1, n + 2), -1), seen=[50], decay=0.5)
    want = p.sum((0, 1))
    want[:n - r] += 0.5 * acc[0, 0, :n - r]
    np.testing.assert_allclose(new[0, 0, :n], want, atol=1e-12)
    np.testing.assert_array_equal(new[0, 0, n:], acc[0, 0, n:])
    assert pos[0, 0].tolist() == [-1] * 5 + [46, 47, 48, 49] + [-1] * 2
    np.testing.assert_allclose(evict.kv_weigh(q, lse, k, [n], acc, pos, decay=0.0)[0][0, 0, :n].sum(), 2 * r)
    # a path is the chain of its nodes
    a, _, _ = evict.kv_weigh(q[:, :, [3, 0, 2, 1]], lse[:, :, [3, 0, 2, 1]], k, [n], acc, pos, path=[[1, 3, 2, 0]], decay=0.5)
    np.testing.assert_allclose(a, new)


def test_eviction_keeps_the_best_and_moves_the_least():
    acc = np.array([5.0, 1.0, 3.0, np.nan, 4.0, 0.5, 3.0, 2.0])
    pos = np.array([0, 4, 2, 3, 1, 5, 6, 7])
    # protected: position 0 (place 0), positions 6 and 7 (places 6, 7); then 4.0 and the first 3.0
    assert evict.kept_places(acc, pos, 8, 5, 1, 2, 8) == [0, 6, 2, 7, 4]
    assert evict.kept_places(acc, pos, 8, 2, 0, 0, 8) == [0, 4]
    assert evict.kept_places(acc, pos, 8, 1, 0, 1, 8) == [7]
    assert evict.kept_places(acc, pos, 4, 4, 0, 0, 8) == [0, 1, 2, 3]
    assert evict.kept_places(np.zeros(4), np.arange(4), 4, 3, 0, 0, 4) == [0, 1, 2]


@pytest.mark.parametrize("into", [False, True])
def test_a_paged_eviction_is_the_contiguous_one_through_the_table(into):
    rng = np.random.default_rng(3)
    B, H, D, bs, width = 2, 3, 4, 2, 4
    table = rng.permutation(B * width).reshape(B, width)
    pool = lambda c: np.stack([c[b, :, j * bs:(j + 1) * bs] for b, j in sorted(((b, j) for b in range(B) for j in range(width)),  # noqa: E731
                                                                              key=lambda e: table[e])])
    k, v = rng.standard_normal((B, H, 8, D)), rng.standard_normal((B, H, 8, D))
    acc, pos = rng.random((B, H, 8)), np.tile(np.arange(8), (B, H, 1))
    args = dict(budget=3, sink=1, recent=1)
    if not into:
        k1, v1, a1, p1, n1 = evict.kv_evict(k, v, acc, pos, np.array([8, 2]), **args)
        k2, v2, a2, p2, n2 = evict.kv_evict(pool(k), pool(v), acc, pos, np.array([8, 2]), table=table, **args)
        np.testing.assert_array_equal(pool(k1), k2)
        np.testing.assert_array_equal(pool(v1), v2)
    else:
        zero = [np.zeros((B, H, 4, D)), np.zeros((B, H, 4, D)), np.zeros((B, H, 4)), np.zeros((B, H, 4), dtype=int)]
        k1, v1, a1, p1, n1 = evict.kv_evict(k, v, acc, pos, np.array([8, 2]), out=zero, **args)
        more = np.concatenate([pool(k), np.zeros((4, H, bs, D))]), np.concatenate([pool(v), np.zeros((4, H, bs, D))])
        out_table = np.array([[8, 11], [9, 10]])
        k2, v2, a2, p2, n2 = evict.kv_evict(*more, acc, pos, np.array([8, 2]), table=table, out=zero[2:], out_table=out_table, **args)
        np.testing.assert_array_equal(k2[out_table].transpose(0, 2, 1, 3, 4).reshape(B, H, 4, D), k1)
        np.testing.assert_array_equal(k2[:8], pool(k))
    np.testing.assert_array_equal(a1, a2)
    np.testing.assert_array_equal(p1, p2)
    assert n1.tolist() == n2.tolist() == [3, 2]


def test_attention_does_not_depend_on_the_order_that_eviction_leaves():
    rng = np.random.default_rng(4)
    H, n, D, T = 1, 6, 4, 1
    tree = oracle.tree_encode(np.array([-1]), np.array([0]))
    k, v = rng.standard_normal((1, H, n, D)), rng.standard_normal((1, H, n, D))
    acc, pos = rng.random((1, H, n)), np.arange(n)[None, None]
    k1, v1, _, p1, m = evict.kv_evict(k, v, acc, pos, np.array([n]), 4)
    kept = np.sort(p1[0, 0, :4])
    q, kt, vt = (rng.standard_normal((1, H, T, D)).astype(np.float32) for _ in range(3))
    f = lambda x: np.ascontiguousarray(x, dtype=np.float32)  # noqa: E731
    a = oracle.tree_attention(q, f(k1), f(v1), m, kt, vt, tree, "f32")[0]
    b = oracle.tree_attention(q, f(k[:, :, kept]), f(v[:, :, kept]), m, kt, vt, tree, "f32")[0]
    np.testing.assert_allclose(a, b, atol=1e-12)
