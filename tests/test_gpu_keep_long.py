"""i8_kv_keep of branches of more than 64 rows: every block that they touch is
scaled once, by all tokens that come into it, wherever in a block the tree
begins.  Bit for bit against the oracle."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw

from test_gpu_kv import Case
from test_gpu_tree import kept_cache

pytestmark = pytest.mark.gpu


def some(rng, rows, count, width):
    path = np.full(width, -1, np.int32)
    path[:count] = np.sort(rng.choice(rows, count, replace=False))
    return path


@pytest.mark.parametrize("d, heads", [(128, 1), (64, 3)])
@pytest.mark.parametrize("rows, prev, count", [
    (300, 10, 120), (300, 63, 65), (512, 1, 300), (512, 127, 400), (200, 33, 64), (200, 31, 66), (512, 64, 200),
    (400, 37, 129), (512, 50, 511), (100, 5, 70)])
def test_long_branches(d, heads, rows, prev, count):
    for seed in range(4):
        s = Case(tw, [d, rows, count, seed], d, heads, [rows], [prev])
        s.scales *= np.exp2(s.rng.integers(-6, 7, s.scales.shape)).astype(np.float32)
        if seed == 3:
            s.scales[s.rng.random(s.scales.shape) < 0.3] = 0
        kept_cache(s, some(s.rng, rows, count, count + seed)[None])


def test_a_batch_of_them():
    """Beside short ones, and one whose path ends early because it does not ascend."""
    new, prev, counts = [512, 9, 300, 0, 130, 512], [17, 60, 64, 5, 100, 3], [450, 5, 100, 0, 80, 200]
    for seed in range(3):
        s = Case(tw, [77, seed], 64, 2, new, prev)
        s.scales *= np.exp2(s.rng.integers(-6, 7, s.scales.shape)).astype(np.float32)
        paths = np.stack([some(s.rng, n, c, 460) for n, c in zip(new, counts)])
        paths[5, 150] = paths[5, 149]
        kept_cache(s, paths)


def test_a_branch_that_begins_in_front_of_the_cache():
    """Rows in front of position 0 are not there; blocks that the table lacks are passed over."""
    s = Case(tw, 83, 64, 2, [400], [20])
    s.scales *= np.exp2(s.rng.integers(-6, 7, s.scales.shape)).astype(np.float32)
    s.lens[0] = 330                                     # rows 0 to 69 in front of position 0
    path = some(s.rng, 400, 250, 250)[None]
    kept_cache(s, path)
    for gone in (0, 1, 4):
        table = s.table.copy()
        table[0, gone] = -1
        kept_cache(s, path, table)


def test_scales_from_the_smallest_numbers():
    """Blocks whose scale has to grow from below fp32's normal numbers to ordinary sizes."""
    for seed in range(4):
        s = Case(tw, [91, seed], 64, 2, [200], [50])
        s.scales[s.rng.random(s.scales.shape) < 0.4] = (2.0 ** -149, 1e-42, 2.0 ** -126, 1e-30)[seed]
        kept_cache(s, some(s.rng, 200, 90, 90)[None])
