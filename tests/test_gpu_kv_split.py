"""The int8 path of i8_kv_attend where long sequences are cut into stretches
and their parts joined, at its edges, against the 64-bit oracle.  Every test
asserts the path it covers."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import kv

from test_gpu_kv import Case, dev, host, queries
from test_gpu_kv_tile import attend, exact, path

pytestmark = pytest.mark.gpu

# columns of a tile -> rows, what stands in front of them, key/value heads, query heads
SIZES = {16: ([1, 3], [4000, 5100], 2, 8), 32: ([7, 6], [16700, 16400], 8, 32), 64: ([15, 14], [16400, 16700], 8, 32)}


def make(cols, seed, d=64):
    new, prev, heads, hq = SIZES[cols]
    s = Case(tw, seed, d, heads, new, prev)
    launches = path(s, hq, 0, None)
    assert len(launches) == 1 and launches[0]["cols"] == cols and launches[0]["groups"] > 0, launches
    return s, hq


def check(s, q, window=0, scale=None):
    got = attend(s, q, window, scale)
    want, bound = exact(s, q, window, scale)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)
    return got


@pytest.mark.parametrize("cols", SIZES)
def test_uneven_scales(cols):
    s, hq = make(cols, 600, 128)
    s.scales[:, :, 1] *= (10.0 ** s.rng.uniform(-9, 9, s.scales.shape[:2])).astype(np.float32)
    s.scales[s.table[0, 2]] = 0
    s.scales[s.table[1, 4], :, 1] = 0
    check(s, queries(s, hq))


@pytest.mark.parametrize("cols", SIZES)
def test_missing_blocks(cols):
    s, hq = make(cols, 610)
    n = -(-int(s.lens[0]) // 64)
    s.table[0, [0, 3, 4, 5, 40, n - 1]] = -1, 10 ** 6, -1, len(s.codes), -2 ** 31, -1
    s.table[0, 10:30] = -1                           # whole stretches of nothing
    check(s, queries(s, hq))
    s.table[1] = -1
    got = check(s, queries(s, hq))
    assert np.all(got[s.cu[1]:] == 0)


@pytest.mark.parametrize("cols", SIZES)
def test_rows_that_see_nothing(cols):
    s, hq = make(cols, 620)
    s.lens[0] = (s.new[0] + 1) // 2
    check(s, queries(s, hq))
    s.lens[1] = 0
    got = check(s, queries(s, hq))
    assert np.all(got[s.cu[1]:] == 0)


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("cols", SIZES)
def test_scales_that_are_not_finite(cols, bad, side):
    s, hq = make(cols, 630)
    q = queries(s, hq)
    want, bound = exact(s, q)
    s.codes[s.table[0, 30], -1, side] = 0
    s.scales[s.table[0, 30], -1, side] = bad
    got = attend(s, q)
    sees = np.zeros(got.shape, bool)
    sees[:s.cu[1], hq - hq // s.heads:] = True
    assert np.array_equal(np.isnan(got), sees)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[~sees])


@pytest.mark.parametrize("cols", SIZES)
def test_queries_that_are_not_finite(cols):
    s, hq = make(cols, 640)
    q = queries(s, hq)
    want, bound = exact(s, q)
    bad = np.zeros(q.shape, bool)
    for t, h, d, x in ((0, 0, 3, np.nan), (s.tokens - 1, 1, 40, np.inf), (1, hq - 1, 63, -np.inf)):
        q[t, h, d] = x
        bad[t, h] = True
    got = attend(s, q)
    assert np.array_equal(np.isnan(got), bad)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[~bad])


@pytest.mark.parametrize("cols", SIZES)
def test_what_is_masked_changes_nothing(cols):
    s, hq = make(cols, 650)
    q = queries(s, hq)
    first = check(s, q)
    for i in range(2):
        last, left = divmod(int(s.lens[i]) - 1, 64)
        for side in (0, 1):
            tail = kv.place(side, s.d)[left + 1:].ravel()
            s.codes[s.table[i, last], :, side][:, tail] = -127
    s.scales[np.setdiff1d(np.arange(len(s.codes)), s.table)] = np.nan
    assert np.array_equal(first, attend(s, q))


@pytest.mark.parametrize("scale", [0.0, -0.05])
@pytest.mark.parametrize("cols", SIZES)
def test_scale(cols, scale):
    s, hq = make(cols, 660)
    check(s, queries(s, hq), scale=scale)
