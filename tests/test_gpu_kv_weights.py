"""How far down the attention's weights keep their digits: one token that
outweighs all others by 2^k and has nothing in half of the dims, where the
result is what the others leave."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import kv

from test_gpu_kv import Case
from test_gpu_kv_tile import LONG, assert_kind, attend, exact

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [10, 20, 23, 26])
@pytest.mark.parametrize("kind, heads, hq, new, prev, max_len", [
    ("split", 1, 4, [200], [500], LONG), ("whole", 16, 64, [600], [1500], None),
])
def test_small_weights_beside_a_large_one(kind, heads, hq, new, prev, max_len, k):
    s = Case(tw, 700 + k, 64, heads, new, prev)
    s.codes[:, :, 0] = 0
    s.scales[:] = 0.02
    first, at = s.table[0, 0], kv.place(0, 64)[7]
    s.codes[first, :, 0][:, at] = 100                       # score 100 * 0.02 * 64 * scale = k ln 2
    s.codes[first, :, 1][:, kv.place(1, 64)[7, :32]] = 0
    s.codes[:, :, 1] = np.abs(s.codes[:, :, 1])             # the others add up
    scale = k * np.log(2.0) / 128
    q = np.ones((s.tokens, hq, 64), np.float32)
    assert_kind(kind, s, hq, 0, max_len)
    got = attend(s, q, scale=scale, max_len=max_len)
    want, bound = exact(s, q, scale=scale)
    err = np.abs(got - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + bound)
    # the bound leaves no room for weights that have vanished
    assert np.all(bound[..., :32] < 0.25 * np.abs(want[..., :32]))
