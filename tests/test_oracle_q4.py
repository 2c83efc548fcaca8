"""The 4-bit oracle against its definition, by hand (no GPU)."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import q4


@pytest.mark.parametrize("n, k, group", [(0, 128, 128), (1, 0, 32), (16, 128, 32), (17, 640, 64), (4096, 12288, 128)])
def test_sizes(n, k, group):
    assert tw.q4_packed_bytes(n, k, group) == q4.packed_bytes(n, k, group) >= 0


@pytest.mark.parametrize("n, k, group", [(-1, 128, 32), (1, 64, 32), (1, -128, 32), (1, 128, 16), (1, 128, 256),
                                         (1, 128, 0)])
def test_bad_sizes(n, k, group):
    assert tw.q4_packed_bytes(n, k, group) == q4.packed_bytes(n, k, group) == -1


def test_places_by_hand():
    """Single weights and scales at places worked out from the layout."""
    t = np.zeros((18, 640), np.int64)
    s = np.zeros((18, 10), np.float16)
    t[17, 128 * 4 + 32 * 3 + 8 * 2 + 5] = -3          # tile 1, row 1, block 4, c 3, g 2, i 5
    s[17, 9] = 1.0                                    # block 4, second half: the last, narrower k-tile
    s[0, 3] = 2.0                                     # block 1, second half
    blob = q4.pack(t, s)
    words, scales = blob[:32 * 640 // 2].view(np.uint32), blob[32 * 640 // 2:].view(np.float16)
    assert np.flatnonzero(words).tolist() == [(5 + 4) * 256 + (2 * 16 + 1) * 4 + 3]
    assert words.max() == 13 << (16 + 8)
    assert {int(e): float(scales[e]) for e in np.flatnonzero(scales)} == {
        ((5 + 4) * 16 + 1) * 2 + 1: 1.0, (1) * 2 + 1: 2.0}


def test_product():
    rng = np.random.default_rng(5)
    t, s = rng.integers(-8, 8, (3, 128)), rng.uniform(0.1, 1, (3, 4)).astype(np.float16)
    x = rng.normal(size=(2, 128))
    want = [[sum(float(t[n, k]) * float(s[n, k // 32]) * x[m, k] for k in range(128)) for n in range(3)] for m in range(2)]
    assert np.allclose(q4.gemv(t, s, x)[0], want, rtol=1e-12)
    q = rng.integers(-127, 128, (2, 128))
    assert np.allclose(q4.gemv_i8(t, s, q, [0.5, 2.0])[0], q4.gemv(t, s, q * [[0.5], [2.0]])[0], rtol=1e-12)
