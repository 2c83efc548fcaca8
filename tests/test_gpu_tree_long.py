"""Attention of trees in the 128-column tiles where a workgroup has more than
64 blocks of a unit: keys that score far above all before them stand in the
blocks with which each further 64 begin, beside V scales that grow there."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import kv, tree

from test_gpu_kv import Case, dev
from test_gpu_tree import forest, host

pytestmark = pytest.mark.gpu

LONG = 10 ** 6


def shared(seed, d, heads, hq, new, prev):
    """Sequences that read the blocks of one, each with rows of its own, and queries that lean one way."""
    s = Case(tw, [seed, d], d, heads, [max(new)], [max(prev)])
    s.new, s.prev = np.array(new), np.array(prev)
    s.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s.lens = (s.new + s.prev).astype(np.int32)
    s.table = np.repeat(s.table, len(new), 0)
    s.tokens = int(s.cu[-1])
    return s, kv.bf16(s.rng.normal(size=(s.tokens, hq, d)) * 1.5 + 1.0)


def raise_key(s, position, size, v_scale):
    """The key at this position points the way that the queries lean, scoring about 1000 `size`; its block's scales
    (the block's other keys score with 130 `size` or so, no more than others unless `size` is large)."""
    block = s.table[0, position // 64]
    s.codes[block, :, 0][:, kv.place(0, s.d)[position % 64]] = 127
    s.scales[block, :, 0] = size * 8 / s.d ** 0.5
    s.scales[block, :, 1] = v_scale


def check(s, q, max_len, cut, seqs, kv_heads):
    import torch
    hq = q.shape[1]
    g = hq // s.heads
    p = tw.i8_kv_attend_tree_config(s.tokens, hq, s.heads, s.d, len(s.new), s.table.shape[1], max_len)
    assert p["cols"] == 128 and (p["groups"] > 0) == cut, p
    if cut:                                              # units alike: on average a workgroup has more than 64 blocks
        units = len(s.new) * s.heads * -(-s.new[0] * g // 128)
        assert set(s.new) == {s.new[0]} and set(s.lens) == {s.lens[0]}
        assert units * (s.lens[0] // 64 + 1) > 64 * p["groups"]
    words = -(-max(s.new) // 64)
    c, b = s.device()
    m, _ = tw.draft_tree_mask(b, dev(forest(s.rng, s.new)), words)
    got = host(tw.i8_kv_attend_tree(c, b, dev(q, torch.bfloat16), m, max_len=max_len))
    assert np.sum(~np.isfinite(got)) == 0
    masks = host(m).view(np.uint64)
    for i in seqs:
        rows = slice(s.cu[i], s.cu[i + 1])
        for h in kv_heads:
            one = kv.Cache(s.codes[:, h:h + 1], s.scales[:, h:h + 1])
            mine = q[rows, h * g:(h + 1) * g]
            want, bound = tree.attend(one, np.array([0, s.new[i]]), s.lens[i:i + 1], s.table[i:i + 1], mine,
                                      s.d ** -0.5, masks[rows])
            off = np.abs(got[rows, h * g:(h + 1) * g] - want)
            assert np.all(off <= 2.0 ** -8 * np.abs(want) + bound), (i, h, off.max())


@pytest.mark.parametrize("d", [64, 128])
def test_whole_units(d):
    s, q = shared(1, d, 8, 32, [24] * 140, [40] * 139 + [8900])
    for position, size, v_scale in ((64 * 64 + 5, 0.03, 0.08), (64 * 128 + 60, 0.06, 0.3)):
        raise_key(s, position, size, v_scale)
    check(s, q, 20000, False, (3, 139), (0, 5))


@pytest.mark.parametrize("d", [64, 128])
def test_cut_units(d):
    """Chunks of 70 blocks: their second 64 begin at blocks 64 and 134."""
    s, q = shared(2, d, 8, 32, [24] * 40, [8900] * 40)
    for position, size, v_scale in ((64 * 64, 0.03, 0.08), (64 * 128 + 60, 0.06, 0.3), (64 * 134 + 63, 0.1, 0.02)):
        raise_key(s, position, size, v_scale)
    check(s, q, None, True, (0, 39), (0, 7))


@pytest.mark.parametrize("prev", [64 * 64 + 3, 64 * 128 - 9])
def test_blocks_with_masks(prev):
    """The raised key is the root's own, in block 64 or in the block in front of block 128, beside one in block 128
    that only some rows see."""
    s, q = shared(3, 64, 8, 32, [24] * 140, [40] * 139 + [prev])
    raise_key(s, prev, 0.02, 0.08)
    raise_key(s, prev + 20, 0.03, 0.2)
    check(s, q, 20000, False, (139,), (2, 7))


@pytest.mark.parametrize("gone", [range(10, 30), range(64, 130)])
def test_blocks_that_are_not_there(gone):
    """Blocks that the table does not have: 64 that follow are not 64 that are there."""
    s, q = shared(4, 64, 8, 32, [24] * 140, [40] * 139 + [8900])
    first = 64 if gone[-1] < 64 else 130
    raise_key(s, 64 * first + 9, 0.03, 0.1)
    raise_key(s, 64 * 136 + 9, 0.04, 0.01)
    s.table[-1, gone] = -1
    check(s, q, 20000, False, (139,), (1,))
