"""The tree oracle against cases worked out by hand (no GPU)."""
import numpy as np

from oracle import kv, tree

#            0
#        1       2         3 stands apart: no row continues it
#      4   5     6
#      7
PARENT = [-1, 0, 0, -1, 1, 1, 2, 4]


def test_masks_and_positions():
    cu, lens = [1, 9], [20]
    parent = np.array([5] + PARENT + [0])
    m, pos = tree.mask(cu, lens, parent, 1, np.full((10, 1), 99, np.uint64), np.full(10, -7))
    assert m[:, 0].tolist() == [99, 1, 0b11, 0b101, 0b1000, 0b10011, 0b100011, 0b1000101, 0b10010011, 99]
    assert pos.tolist() == [-7, 12, 13, 13, 12, 14, 14, 14, 15, -7]


def test_odd_parents_count_as_none():
    m, _ = tree.mask([0, 4], [4], np.array([3, 1, 7, -5]), 1, np.zeros((4, 1), np.uint64), np.zeros(4))
    assert m[:, 0].tolist() == [1, 2, 4, 8]


def test_accepted_branch():
    token = np.array([10, 11, 12, 13, 14, 15, 16, 17])
    target = np.array([11, 15, 0, 0, 0, 99, 0, 0])
    path, count, following = tree.accept([0, 8], np.array(PARENT), token, target, 5)
    assert path.tolist() == [[0, 1, 5, -1, -1]] and count.tolist() == [3] and following.tolist() == [99]
    path, count, following = tree.accept([0, 8], np.array(PARENT), token, target, 2)
    assert path.tolist() == [[0, 1]] and count.tolist() == [2] and following.tolist() == [15]


def test_kept_entries():
    assert tree.kept([0, 2, 2, 3], 8) == [0, 2]
    assert tree.kept([0, 9, 3], 8) == [0]
    assert tree.kept([-1, 3], 8) == []
    assert tree.kept([3, 1], 8) == [3]


def test_tokens_move_within_and_across_blocks():
    rng = np.random.default_rng(3)
    codes = rng.integers(-127, 128, (3, 1, 2, 64 * 64)).astype(np.int8)
    scales = np.array([[[0.5, 0.25]], [[2.0, 0.25]], [[1.0, 1.0]]], np.float32)
    c = kv.Cache(codes, scales)
    before = [[c.tokens(b, 0, side).astype(float) for side in (0, 1)] for b in range(3)]
    # rows 0..9 at slots 60..69 of blocks 2 -> 0 -> 1: (table) block 0 is 0, block 1 is 1
    lens = tree.keep(c, [0, 10], [70], np.array([[0, 1]]), 10, [[0, 2, 5]])
    assert lens.tolist() == [63]
    # slot 61 takes slot 62 (same block), slot 62 takes slot 65 - 64 = 1 of block 1
    g = 0
    while np.abs(before[1][0][1]).max() * 2.0 > 127 * 0.5 * 2 ** g:
        g += 1
    k = c.tokens(0, 0, 0)
    assert c.scales[0, 0, 0] == 0.5 * 2 ** g
    assert np.array_equal(k[61], np.rint(before[0][0][62] / 2 ** g))
    assert np.array_equal(k[62], np.clip(np.rint(before[1][0][1] * 2.0 / c.scales[0, 0, 0]), -127, 127))
    v = c.tokens(0, 0, 1)
    assert c.scales[0, 0, 1] == 0.25 and np.array_equal(v[62], before[1][1][1]) and np.array_equal(v[0], before[0][1][0])
    assert np.array_equal(c.tokens(1, 0, 0), before[1][0])


def test_a_scale_grows_by_any_power_of_two():
    """From fp32's smallest numbers to ordinary ones: 2^g itself passes fp32."""
    codes = np.full((2, 1, 2, 64 * 64), 100, np.int8)
    for small in (2.0 ** -149, 1e-42, 1e-30):
        scales = np.array([[[small, 0.5]], [[2.0, 2.0]]], np.float32)
        c = kv.Cache(codes.copy(), scales)
        tree.keep(c, [0, 10], [70], np.array([[0, 1]]), 10, [[0, 9]])     # slot 61 takes slot 69
        g = np.log2(c.scales[0, 0] / scales[0, 0].astype(np.float64))
        assert np.array_equal(g, np.rint(g)) and np.all(127 * c.scales[0, 0].astype(np.float64) >= 200)
        assert np.all(127 * c.scales[0, 0] / 2 < 200)
        assert np.all(c.tokens(0, 0, 0)[61] == np.rint(200 / np.float32(c.scales[0, 0, 0])))
