"""Pins of the block-sparse oracle against closed forms and independent statements."""

import numpy as np
import pytest

import oracle as orc
from oracle import sparse as sp


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_table_of_one_axis_is_the_complex_exponential():
    pos = np.array([[0, 1, -3, 1 << 30]])
    t, turns = sp.rope_table(pos, [8], base=100.0)
    for j in range(4):
        np.testing.assert_allclose(t[:3, j, 0] + 1j * t[:3, j, 1], np.exp(1j * pos[0, :3] * 100.0 ** (-j / 4)), atol=1e-15)
    np.testing.assert_allclose(t[0], [[1, 0]] * 4)
    assert turns.shape == (4, 4)


def test_axes_stand_side_by_side():
    pos = rng(0).integers(0, 50, (3, 7))
    t, _ = sp.rope_table(pos, [4, 6, 2])
    for a, (lo, hi) in enumerate([(0, 2), (2, 5), (5, 6)]):
        np.testing.assert_array_equal(t[:, lo:hi], sp.rope_table(pos[a:a + 1], [[4, 6, 2][a]])[0])


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(halves):
    r = rng(1)
    x, z = r.standard_normal((2, 1, 1, 16))
    def at(v, pos):
        return sp.norm_rope(v, None, sp.rope_table([[pos]], [16])[0], halves, norm=False)[0][0, 0]
    np.testing.assert_allclose(np.linalg.norm(at(x, 77)), np.linalg.norm(x))
    # the product of two rotated rows depends on the difference of their positions alone
    np.testing.assert_allclose(at(x, 12) @ at(z, 5), at(x, 107) @ at(z, 100), rtol=1e-12)


def test_norm_gives_weighted_unit_mean_square():
    x = rng(2).standard_normal((2, 3, 24)) * 5
    w = rng(3).standard_normal(24)
    y, _ = sp.norm_rope(x, None, None, eps=0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1.0)
    np.testing.assert_allclose(sp.norm_rope(x, w, None, eps=0.0)[0], y * w)


def test_block_means_of_a_short_last_block():
    y = np.arange(130.0)[None, :, None]
    np.testing.assert_allclose(sp.block_means(y, 64)[0, :, 0], [31.5, 95.5, 128.5])


def test_selection_by_hand():
    # scores of one query block: 1, 3, 3, 2, nan, 0
    qm = np.array([[[1.0, 0, 0, 0]]])
    km = np.zeros((1, 6, 4))
    km[0, :, 0] = [2, 6, 6, 4, np.nan, 0]
    idx, count = sp.block_select(qm, km, 3)
    np.testing.assert_array_equal(idx[0, 0], [1, 2, 3])
    np.testing.assert_array_equal(sp.block_select(qm, km, 1)[0][0, 0], [1])            # equal scores: the lower index
    np.testing.assert_array_equal(sp.block_select(qm, km, 3, 1, 1)[0][0, 0], [0, 1, 5])
    idx, count = sp.block_select(qm, km, 4, margin=0.5)
    np.testing.assert_array_equal(idx[0, 0], [1, 2, -1, -1])
    assert count[0, 0] == 2


def test_all_blocks_listed_is_full_attention_in_any_order():
    r = rng(4)
    q, k, v = r.standard_normal((2, 150, 8)), r.standard_normal((1, 200, 8)), r.standard_normal((1, 200, 8))
    for block, perm in ((64, [0, 1, 2, 3]), (64, [3, 1, 0, 2]), (128, [1, 0])):
        idx = np.broadcast_to(np.array(perm, np.int32), (2, 2, len(perm)))
        O, L, _, _ = sp.block_sparse_attention(q, k, v, idx, np.full((2, 2), len(perm)), block)
        for h in range(2):
            s = q[h] @ k[0].T / np.sqrt(8)
            p = np.exp(s)
            np.testing.assert_allclose(O[h], p @ v[0] / p.sum(1, keepdims=True), atol=1e-12)
            np.testing.assert_allclose(L[h], np.log(p.sum(1)), atol=1e-12)


def test_states_of_disjoint_lists_compose_to_their_union():
    r = rng(5)
    q, k, v = r.standard_normal((1, 10, 8)), r.standard_normal((1, 300, 8)), r.standard_normal((1, 300, 8))
    def state(blocks):
        idx = np.array(blocks, np.int32)[None, None]
        O, L, _, _ = sp.block_sparse_attention(q, k, v, idx, np.array([[len(blocks)]]), 64)
        return O[0], L[0]
    O, L = orc.compose_n([state([0, 3]), state([1, 2, 4])])
    full = state([0, 1, 2, 3, 4])
    np.testing.assert_allclose(O, full[0], atol=1e-12)
    np.testing.assert_allclose(L, full[1], atol=1e-12)


def test_nothing_listed_is_the_empty_state_and_twice_counts_twice():
    r = rng(6)
    q, k, v = (r.standard_normal((1, 5, 8)) for _ in range(3))
    O, L, _, _ = sp.block_sparse_attention(q, k, v, np.full((1, 1, 2), -1), np.array([[0]]), 64)
    assert not O.any() and np.all(np.isneginf(L))
    one = sp.block_sparse_attention(q, k, v, np.array([[[0, 0]]]), np.array([[1]]), 64)
    two = sp.block_sparse_attention(q, k, v, np.array([[[0, 0]]]), np.array([[2]]), 64)
    np.testing.assert_allclose(one[0], two[0])
    np.testing.assert_allclose(two[1], one[1] + np.log(2))
