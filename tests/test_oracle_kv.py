"""The oracle of the paged int8 cache against what can be said by hand (no GPU)."""
import numpy as np
import pytest

from oracle import kv


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("side", [0, 1])
def test_every_byte_of_a_block_has_one_place(side, d):
    assert sorted(kv.place(side, d).ravel()) == list(range(64 * d))


def test_places_by_hand():
    # K: token 17, dim 70 of D = 128 is t 1, r 1, s 1, g 0, b 6
    assert kv.place(0, 128)[17, 70] == (((1 * 2 + 1) * 4 + 0) * 16 + 1) * 16 + 6
    # V: token 39 is t 2, g 1, i 3; dim 33 is u 2, r 1
    assert kv.place(1, 64)[39, 33] == ((2 * 4 + 1) * 16 + 1) * 16 + 4 * 2 + 3


def test_rotation_keeps_dot_products_of_equal_distance():
    rng = np.random.default_rng(1)
    f = 1e6 ** (-np.arange(0, 64, 2) / 64)
    a, b = rng.normal(size=(2, 1, 1, 64))
    for inter in (False, True):
        turn = lambda x, p: kv.transform(x, None, 0.0, f, inter, [p])[0, 0]
        assert turn(a, 907) @ turn(b, 900) == pytest.approx(turn(a, 7) @ turn(b, 0), abs=1e-9)
        assert np.allclose(turn(a, 0), a[0, 0])


def test_norm_by_hand():
    x = np.array([[[3.0, 4.0] * 32]])
    y = kv.transform(x, np.full(64, 2.0), 0.0, None, False, None)
    assert np.allclose(y[0, 0, :2], np.array([3.0, 4.0]) * 2 / np.sqrt(12.5))


def fresh(blocks=3, heads=1, d=64, fill=0):
    return kv.Cache(np.full((blocks, heads, 2, 64 * d), fill, np.int8), np.zeros((blocks, heads, 2), np.float32))


def test_append_grows_by_doubling():
    c = fresh()
    table = np.array([[2]], np.int32)
    one = np.zeros((1, 1, 64), np.float32)
    one[0, 0, :3] = 127.0, 5.0, -3.0
    c.append([0, 1], [1], table, one, one)
    assert c.scales[2, 0, 0] == 1.0 and list(c.tokens(2, 0, 0)[0, :3]) == [127, 5, -3]
    c.append([0, 1], [2], table, one * 2.5, one)         # 317.5 needs scale 4
    assert c.scales[2, 0, 0] == 4.0 and c.scales[2, 0, 1] == 1.0
    assert list(c.tokens(2, 0, 0)[0, :3]) == [32, 1, -1]             # 31.75, 1.25, -0.75
    assert list(c.tokens(2, 0, 0)[1, :3]) == [79, 3, -2]             # 79.375, 3.125, -1.875
    c.append([0, 1], [1], table, one / 2, one)           # the first slot again: a new scale
    assert c.scales[2, 0, 0] == 0.5


def test_repeated_growth_stays_below_one_step():
    rng = np.random.default_rng(2)
    c = fresh()
    table = np.array([[0]], np.int32)
    rows = (rng.normal(size=(64, 1, 1, 64)) * 1.4 ** np.arange(64)[:, None, None, None]).astype(np.float32)
    for p in range(64):
        c.append([0, 1], [p + 1], table, rows[p], rows[p])
    k = c.read([0, 64], [64], table, 64)[0]
    assert np.abs(k - rows[:, 0]).max() < c.scales[0, 0, 0]


def test_attend_by_hand():
    c = fresh(fill=1)
    c.scales[:] = 0.5
    q = np.zeros((2, 2, 64), np.float32)
    out, _ = kv.attend(c, [0, 2], [2], np.array([[1]], np.int32), q, 1.0)
    assert np.all(out == 0.5)
    out, _ = kv.attend(c, [0, 2], [1], np.array([[1]], np.int32), q, 1.0)    # the first row stands before the start
    assert np.all(out[0] == 0) and np.all(out[1] == 0.5)
    out, _ = kv.attend(c, [0, 2], [2], np.array([[7]], np.int32), q, 1.0)    # a block that is not there
    assert np.all(out == 0)
