"""Pins of the rotation oracle (CPU): complex multiplication, the relative-position
property, the place of appended tokens, and what is left out."""

import numpy as np
import pytest

import oracle
from oracle import rope


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 8), (16, 6), (10, 0)])
def test_rotation_is_complex_multiplication(interleaved, D, rot):
    rng = np.random.default_rng(D + rot)
    x = rng.standard_normal((3, D))
    freq = rng.uniform(0, 1, rot // 2)
    y = rope.rotate(x, 37, freq, interleaved)
    z = x[:, 0:rot:2] + 1j * x[:, 1:rot:2] if interleaved else x[:, :rot // 2] + 1j * x[:, rot // 2:rot]
    w = y[:, 0:rot:2] + 1j * y[:, 1:rot:2] if interleaved else y[:, :rot // 2] + 1j * y[:, rot // 2:rot]
    np.testing.assert_allclose(w, z * np.exp(37j * freq), atol=1e-13)
    np.testing.assert_array_equal(y[:, rot:], x[:, rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_scores_depend_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(5)
    q, k, freq = rng.standard_normal(16), rng.standard_normal(16), rng.uniform(0, 1, 8)
    dot = lambda a, b: rope.rotate(q, a, freq, interleaved) @ rope.rotate(k, b, freq, interleaved)  # noqa: E731
    np.testing.assert_allclose([dot(9, 4), dot(1009, 1004)], dot(5, 0), atol=1e-11)


def test_a_paged_append_is_the_contiguous_one_through_the_table():
    rng = np.random.default_rng(6)
    B, H, D, bs, width = 3, 2, 4, 3, 4
    start, L = np.array([1, 5, 5, 8]), np.array([2, 0, 7])
    k, v, q = rng.standard_normal((10, H, D)), rng.standard_normal((10, H, D)), rng.standard_normal((10, 3, D))
    table = rng.permutation(B * width).reshape(B, width)
    kc, vc = rng.standard_normal((B, H, bs * width, D)), rng.standard_normal((B, H, bs * width, D))

    def pool(c):
        p = np.zeros((B * width, H, bs, D))
        for b in range(B):
            for j in range(width):
                p[table[b, j]] = c[b, :, j * bs:(j + 1) * bs]
        return p
    freq = np.array([1.0, 0.1])
    q1, k1, v1, w1 = rope.kv_append(q, k, v, start, L, kc, vc, freq, base=11)
    q2, k2, v2, w2 = rope.kv_append(q, k, v, start, L, pool(kc), pool(vc), freq, base=11, table=table)
    np.testing.assert_array_equal(pool(k1), k2)
    np.testing.assert_array_equal(pool(v1), v2)
    np.testing.assert_array_equal(q1, q2)
    assert w1.tolist() == w2.tolist() == [False] + [True] * 7 + [False] * 2
    np.testing.assert_allclose(k1[0, :, 3], rope.rotate(k[2], 14, freq, False))
    np.testing.assert_array_equal(k1[:, :, 10:], kc[:, :, 10:])


def test_what_does_not_fit_is_left_out():
    k = np.ones((4, 1, 4))
    cache = np.zeros((2, 1, 3, 4))
    _, kc, _, w = rope.kv_append(k, k, k, [0, 2, 4], [2, -1], cache, cache, [0.5])
    assert not kc.any() and not w.any()
    table = np.array([[0, 9]])
    _, kc, _, w = rope.kv_append(k, k, k, [0, 4], [1], cache, cache, [0.5], table=table)
    assert w.tolist() == [True, True, False, False] and not kc[1].any()


def test_a_node_is_turned_as_on_its_path():
    parent = [-1, 0, 0, 1, 3]
    tree = oracle.tree_encode(parent, None)
    rng = np.random.default_rng(8)
    q, k, v = rng.standard_normal((2, 5, 3, 6)), rng.standard_normal((2, 5, 1, 6)), rng.standard_normal((2, 5, 1, 6))
    freq = np.array([1.0, 0.3, 0.01])
    qo, ko, vo = rope.tree_rope(q, k, v, [4, 9], tree["depth"], freq, base=2)
    path = [0, 1, 3, 4]
    for b, L in enumerate([4, 9]):
        _, kc, _, _ = rope.kv_append(q[b, path], k[b, path], v[b, path], [0, 4], [L], np.zeros((1, 1, 20, 6)),
                                     np.zeros((1, 1, 20, 6)), freq, base=2)
        np.testing.assert_allclose(ko[b][:, path], kc[0, :, L:L + 4], atol=1e-14)
    np.testing.assert_array_equal(vo, np.moveaxis(v, 1, 2))
    np.testing.assert_allclose(qo[1, :, 2], rope.rotate(q[1, 2], 12, freq, False))


def test_offsets_outside_the_rows_leave_the_sequence_out():
    r = np.random.default_rng(8)
    q, k, v = r.standard_normal((3, 2, 4)), r.standard_normal((3, 1, 4)), r.standard_normal((3, 1, 4))
    kc, vc = r.standard_normal((2, 1, 9, 4)), r.standard_normal((2, 1, 9, 4))
    freq = np.array([0.5, 0.1])
    for start, left_out in (([0, 1, 5], 1), ([-2, 1, 3], 0)):
        out, k2, v2, written = rope.kv_append(q, k, v, start, [2, 3], kc, vc, freq)
        np.testing.assert_array_equal(k2[left_out], kc[left_out])
        np.testing.assert_array_equal(v2[left_out], vc[left_out])
        s0, s1 = start[1 - left_out], start[2 - left_out]
        np.testing.assert_array_equal(np.flatnonzero(written), np.arange(s0, s1))
        assert (v2[1 - left_out, :, [2, 3][1 - left_out]] == v[s0]).all()
