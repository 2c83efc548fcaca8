"""Trees of drafted tokens on the GPU against the 64-bit oracle
(oracle/tree.py): masks and positions, attention over the cache, the accepted
branch, the cache after it, and the step that they make together."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import kv, tree

from test_gpu_kv import Case, dev, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    assert torch.cuda.is_available()
    tw.lib()


def host(t):
    import torch
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def grow(rng, n, reach=8):
    """Parents of a random tree: each row continues one of the `reach` before it, or now and then nothing."""
    return np.array([-1 if j == 0 or rng.random() < 0.05 else j - 1 - rng.integers(min(j, reach)) for j in range(n)],
                    np.int32).reshape(n)


def forest(rng, new, reach=8):
    return np.concatenate([grow(rng, n, reach) for n in new] + [np.zeros(0, np.int32)]).astype(np.int32)


def batch_of(cu, lens, table=None):
    table = np.zeros((len(lens), 1), np.int32) if table is None else table
    return tw.I8KvBatch(dev(np.asarray(cu, np.int32)), dev(np.asarray(lens, np.int32)), dev(table))


# ---- masks and positions ----
@pytest.mark.parametrize("new, words, reach", [
    ([1], 1, 1), ([64], 1, 1), ([64], 1, 64), ([5, 0, 17, 1], 1, 4), ([65, 3], 2, 9), ([512, 130], 8, 1),
    ([512], 8, 400), ([300, 64, 511], 8, 30), ([100, 20], 1, 3), ([700, 3], 8, 5), ([200], 3, 1)])
def test_masks(new, words, reach):
    import torch
    rng = np.random.default_rng([sum(new), words])
    cu = np.concatenate([[0], np.cumsum(new)]) + 2                 # two rows in front, three behind
    lens = np.array(new) + rng.integers(0, 9000, len(new))
    parent = np.concatenate([[7, 7], forest(rng, new, reach), [0, 1, 2]]).astype(np.int32)
    mask = torch.full((len(parent), words), -5, dtype=torch.int64, device="cuda")
    pos = torch.full((len(parent),), -9, dtype=torch.int32, device="cuda")
    want = tree.mask(cu, lens, parent, words, host(mask).view(np.uint64), host(pos))
    tw.draft_tree_mask(batch_of(cu, lens), dev(parent), words, mask=mask, pos=pos)
    assert np.array_equal(host(mask).view(np.uint64), want[0]) and np.array_equal(host(pos), want[1])


def test_masks_of_odd_input():
    """Parents that are no earlier row, lengths shorter than the rows, sequences behind a descent of cu or outside
    the rows."""
    rng = np.random.default_rng(3)
    parent = rng.integers(-40, 60, 90).astype(np.int32)
    for cu, lens in (([0, 30, 60, 90], [40, 10, -5]), ([0, 40, 20, 90], [99, 99, 99]), ([0, 50, 95], [80, 80]),
                     ([-3, 20, 60], [50, 50])):
        before = np.full((90, 1), 77, np.uint64), np.full(90, 77, np.int32)
        m, p = dev(before[0].view(np.int64)), dev(before[1])
        tw.draft_tree_mask(batch_of(cu, lens), dev(parent), 1, mask=m, pos=p)
        want = tree.mask(cu, lens, parent, 1, *before)
        assert np.array_equal(host(m).view(np.uint64), want[0]) and np.array_equal(host(p), want[1]), cu


# ---- attention ----
def check(s, q, parent=None, masks=None, words=1, scale=None, max_len=None):
    import torch
    c, b = s.device()
    if masks is None:
        m, _ = tw.draft_tree_mask(b, dev(parent), words, mask=torch.zeros(s.tokens, words, dtype=torch.int64, device="cuda"))
        masks = host(m).view(np.uint64)
    else:
        m = dev(masks.view(np.int64))
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    tw.i8_kv_attend_tree(c, b, dev(q, torch.bfloat16), m, scale=scale, max_len=max_len, out=out)
    got = host(out)
    want, bound = tree.attend(kv.Cache(s.codes, s.scales), s.cu, s.lens, s.table, q,
                              s.d ** -0.5 if scale is None else scale, masks)
    none = np.isnan(want).all((1, 2))
    assert np.all(got[none] == 9)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[~none])
    return got


@pytest.mark.parametrize("d, heads, hq", [(128, 2, 8), (64, 1, 3), (128, 1, 1), (64, 2, 32)])
@pytest.mark.parametrize("new, prev, words", [
    ([1], [0], 1), ([8], [512], 1), ([64], [37], 1), ([33, 1, 0, 9], [0, 700, 5, 64], 1), ([70, 12], [1000, 63], 2),
    ([130], [129], 3)])
def test_attend(d, heads, hq, new, prev, words):
    s = Case(tw, [d, hq, sum(new)], d, heads, new, prev, spare_rows=2)
    parent = np.concatenate([forest(s.rng, new), [0, 0]]).astype(np.int32)
    check(s, queries(s, hq), parent, words=words)


LONG = 10 ** 6


@pytest.mark.parametrize("d, heads, hq, new, prev, max_len, cols, cut", [
    (64, 2, 4, [5, 3], [300, 100], None, 16, False),
    (128, 8, 32, [20, 1, 64, 33], [130, 700, 0, 64], None, 16, False),
    (128, 2, 8, [4], [9000], None, 16, True),
    (64, 8, 32, [4, 0, 9, 1, 30], [2000, 10, 7000, 64, 0], LONG, 16, True),
    (64, 1, 4, [200], [500], LONG, 128, True),
    (128, 2, 16, [40, 90], [1100, 3], LONG, 128, True),
    (64, 2, 16, [17, 1, 500, 8], [700, 500, 60, 130], LONG, 128, True),
    (64, 2, 32, [8] * 90 + [0, 3], [(37 * i) % 300 for i in range(92)], LONG, 128, True),
    (64, 8, 32, [24] * 140, [40] * 139 + [9000], 20000, 128, False),
    (64, 1, 4, [1] * 100 + [70], [64 * (i % 9) for i in range(101)], LONG, 16, True),
    (64, 800, 800, [90], [20], LONG, 128, True),
    (64, 2, 8, [2] * 300 + [0, 17], [(29 * i) % 200 for i in range(302)], None, 16, False),
    (64, 2, 32, [8] * 300 + [0, 17], [(29 * i) % 200 for i in range(302)], 2000, 128, False),
])
def test_every_path(d, heads, hq, new, prev, max_len, cols, cut):
    s = Case(tw, [7, sum(new)], d, heads, new, prev)
    c = tw.i8_kv_attend_tree_config(s.tokens, hq, heads, d, len(new), s.table.shape[1], max_len)
    assert c["cols"] == cols and (c["groups"] > 0) == cut, c
    check(s, queries(s, hq), forest(s.rng, new, 12), words=-(-max(new) // 64), max_len=max_len)


@pytest.mark.parametrize("new, prev, max_len", [([40], [1500], 1), ([40], [1500], LONG), ([4], [9000], 64)])
def test_the_hint_is_only_a_hint(new, prev, max_len):
    """Lengths above and far below max_len."""
    s = Case(tw, 13, 64, 1, new, prev)
    check(s, queries(s, 4), forest(s.rng, new), max_len=max_len)


@pytest.mark.parametrize("max_len, cols, cut, more", [(None, 16, False, 0), (20000, 16, True, 0), (LONG, 128, True, 0),
                                                      (None, 16, False, 300)])
def test_attend_up_to_a_descent_of_cu(max_len, cols, cut, more):
    """Sequences in front of the descent as if they were alone, rows of the others left as they were."""
    s = Case(tw, 19, 64, 2, [60, 3], [700, 30], spare_rows=30)
    n = int(s.cu[-1])
    s.cu = np.array([0, 60, n, n - 1, n, 2, n + 20] + [n + 30] * (1 + more), np.int32)
    s.lens = np.array([*s.lens, 64, 64, 500, 500, 500] + [300] * more, np.int32)
    s.table = np.concatenate([s.table, np.resize(s.table, (5 + more, s.table.shape[1]))])
    hq = 32 if cols > 16 else 8
    c = tw.i8_kv_attend_tree_config(s.tokens, hq, 2, 64, len(s.lens), s.table.shape[1], max_len)
    assert c["cols"] == cols and (c["groups"] > 0) == cut, c
    parent = np.concatenate([forest(s.rng, [60, 3]), np.zeros(s.tokens - n, np.int32)]).astype(np.int32)
    check(s, queries(s, hq), parent, max_len=max_len)


@pytest.mark.parametrize("hq, max_len", [(8, 20000), (32, LONG)])
def test_one_workspace_for_many_calls(hq, max_len):
    """Calls of other lengths and rows, one after another and in two captured graphs, over one workspace."""
    import torch
    parts, graphs = [], []
    for i, (new, prev) in enumerate((([64], [3000]), ([9, 40], [50, 2000]))):
        s = Case(tw, 81 + i, 64, 1, new, prev)
        c, b = s.device()
        m, _ = tw.draft_tree_mask(b, dev(forest(s.rng, new)))
        parts.append((c, b, dev(queries(s, hq), torch.bfloat16), m))
    want = [tw.i8_kv_attend_tree(*p, max_len=max_len) for p in parts]
    need = [tw.i8_kv_attend_tree_workspace(p[0], p[1], p[2].shape[0], hq, max_len) for p in parts]
    shared = max(need, key=lambda t: t.numel())
    assert shared.numel() > 0
    for p in parts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = tw.i8_kv_attend_tree(*p, max_len=max_len, workspace=shared)
        graphs.append((g, out))
    for k in (0, 1, 1, 0, 0, 1):
        shared.fill_(255)
        got = tw.i8_kv_attend_tree(*parts[1 - k], max_len=max_len, workspace=shared)
        graphs[k][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[k][1], want[k]) and torch.equal(got, want[1 - k])


def test_a_captured_call_follows_the_lengths():
    """A graph of a cut call replayed with other lengths, rows and masks in the same tensors."""
    import torch
    s = Case(tw, 91, 64, 1, [64], [6000])
    q = queries(s, 16)
    c, b = s.device()
    qd = dev(q, torch.bfloat16)
    m = torch.zeros(64, 1, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = tw.i8_kv_attend_tree(c, b, qd, m, max_len=LONG)
    for rows, length in ((64, 6064), (64, 64), (9, 500), (1, 6064), (33, 4000)):
        s.cu, s.lens = np.array([0, rows], np.int32), np.array([length], np.int32)
        b.cu.copy_(dev(s.cu)), b.lens.copy_(dev(s.lens))
        tw.draft_tree_mask(b, dev(np.concatenate([grow(s.rng, rows), np.zeros(64 - rows, np.int32)]).astype(np.int32)),
                           mask=m)
        out.fill_(9.0)
        g.replay()
        got = host(out)
        want, bound = tree.attend(kv.Cache(s.codes, s.scales), s.cu, s.lens, s.table, q, 64 ** -0.5,
                                  host(m).view(np.uint64))
        assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[:rows]) and np.all(got[rows:] == 9)


@pytest.mark.parametrize("rows, prev, max_len", [(6, 0, None), (6, 500, None), (6, 9000, None), (200, 0, 10 ** 6),
                                                 (200, 300, 10 ** 6)])
def test_any_mask(rows, prev, max_len):
    """Bits at random, rows with none, rows whose own bit is not set, bits behind the row and behind the tree."""
    s = Case(tw, [rows, prev], 64, 1, [rows], [prev])
    words = -(-rows // 64) + 1
    masks = s.rng.integers(0, 2 ** 63, (rows, words), dtype=np.uint64) << np.uint64(1)
    masks[1] = 0
    masks[3] = np.uint64(2 ** 64 - 1)
    got = check(s, queries(s, 4), masks=masks, words=words, max_len=max_len)
    if prev == 0:
        assert np.all(got[1] == 0)


def test_no_words_for_the_last_rows():
    """Rows that no word of the masks reaches are seen by none."""
    s = Case(tw, 17, 64, 1, [150], [90])
    check(s, queries(s, 2), forest(s.rng, [150]), words=1)


def test_a_chain_is_causal_attention():
    """Both calls are within the oracle's bound and half a step of bf16 of it, so within twice that of each other."""
    import torch
    for new, prev, hq, max_len in (([7], [3000], 8, None), ([64, 3], [100, 40], 4, None), ([150], [300], 8, LONG)):
        s = Case(tw, 23, 128, 2, new, prev)
        c, b = s.device()
        q = queries(s, hq)
        chain = np.concatenate([np.arange(-1, n - 1) for n in new]).astype(np.int32)
        m, pos = tw.draft_tree_mask(b, dev(chain), -(-max(new) // 64))
        assert np.array_equal(host(pos), np.concatenate([np.arange(n) + p for n, p in zip(new, prev)]))
        one = host(tw.i8_kv_attend_tree(c, b, dev(q, torch.bfloat16), m, max_len=max_len))
        two = host(tw.i8_kv_attend(c, b, dev(q, torch.bfloat16), max_len=max_len))
        want, bound = tree.attend(kv.Cache(s.codes, s.scales), s.cu, s.lens, s.table, q, 128 ** -0.5,
                                  host(m).view(np.uint64))
        assert np.all(np.abs(one - two) <= 2 * (2.0 ** -8 * np.abs(want) + bound))


PATHS = [(2, None, 16, False), (2, 20000, 16, True), (16, LONG, 128, True)]


def on_path(s, hq, max_len, cols, cut):
    c = tw.i8_kv_attend_tree_config(s.tokens, hq, s.heads, s.d, len(s.lens), s.table.shape[1], max_len)
    assert c["cols"] == cols and (c["groups"] > 0) == cut, c


@pytest.mark.parametrize("hq, max_len, cols, cut", PATHS)
def test_what_is_hidden_has_no_say(hq, max_len, cols, cut):
    """Scales that are not finite, and keys of any size, in places that a row does not see."""
    import torch
    s = Case(tw, 29, 64, 1, [70], [60])                 # rows 4..67 in the second block, 68 and 69 in the third
    on_path(s, hq, max_len, cols, cut)
    q = queries(s, hq)
    parent = np.array([-1, 0, 0, 1] + [3] * 66, np.int32)
    parent[68], parent[69] = 2, 68
    c, b = s.device()
    m, _ = tw.draft_tree_mask(b, dev(parent), 2)
    clean = host(tw.i8_kv_attend_tree(c, b, dev(q, torch.bfloat16), m, max_len=max_len))
    for bad in (np.inf, np.nan, 1e30):
        scales = s.scales.copy()
        scales[s.table[0, 1]] = bad                     # the second block: rows 4 to 67
        c2 = tw.I8KvCache(codes=dev(s.codes), scales=dev(scales))
        got = host(tw.i8_kv_attend_tree(c2, b, dev(q, torch.bfloat16), m, max_len=max_len))
        free = [0, 1, 2, 3, 68, 69]                     # see none of them
        assert np.array_equal(got[free], clean[free]), bad
        if not np.isfinite(bad):
            assert np.isnan(got[4:68]).all()


@pytest.mark.parametrize("hq, max_len, cols, cut", PATHS)
def test_queries_that_are_not_finite(hq, max_len, cols, cut):
    """They spoil their own row and head; one that sees nothing gives zeros all the same."""
    import torch
    s = Case(tw, 31, 64, 1, [50], [0])
    on_path(s, hq, max_len, cols, cut)
    q = queries(s, hq)
    c, b = s.device()
    m, _ = tw.draft_tree_mask(b, dev(grow(s.rng, 50)))
    m[7] = 0
    clean = host(tw.i8_kv_attend_tree(c, b, dev(q, torch.bfloat16), m, max_len=max_len))
    bad = q.copy()
    for row, head, value in ((3, 1, np.nan), (7, 0, np.nan), (20, 0, np.inf), (49, hq - 1, -np.inf)):
        bad[row, head, 5] = value
    got = host(tw.i8_kv_attend_tree(c, b, dev(bad, torch.bfloat16), m, max_len=max_len))
    spoilt = np.zeros((50, hq), bool)
    spoilt[3, 1] = spoilt[20, 0] = spoilt[49, hq - 1] = True
    assert np.isnan(got[spoilt]).all() and np.array_equal(got[~spoilt], clean[~spoilt]) and np.all(got[7] == 0)


@pytest.mark.parametrize("hq, max_len, cols, cut", [(8, None, 16, False), (64, LONG, 128, True)])
def test_blocks_past_32_bits(hq, max_len, cols, cut):
    """A cache of more than 4 GiB whose sequences lie at its end: attended and cut to a branch as in a small one."""
    import torch
    d, heads, new, prev = 128, 8, [40], [300]
    s = Case(tw, 33, d, heads, new, prev)
    on_path(s, hq, max_len, cols, cut)
    c, b = s.device()
    small = c.codes.shape[0]
    far = 34000 - small
    codes = torch.zeros(34000, *c.codes.shape[1:], dtype=torch.int8, device="cuda")
    scales = torch.zeros(34000, *c.scales.shape[1:], device="cuda")
    assert codes.numel() > 2 ** 32
    codes[far:], scales[far:] = c.codes, c.scales
    table = dev(np.where(s.table >= 0, s.table + far, s.table).astype(np.int32))
    c2, b2 = tw.I8KvCache(codes=codes, scales=scales), tw.I8KvBatch(b.cu, b.lens, table)
    m, _ = tw.draft_tree_mask(b, dev(forest(s.rng, new)))
    q = dev(queries(s, hq), torch.bfloat16)
    assert torch.equal(tw.i8_kv_attend_tree(c, b, q, m, max_len=max_len),
                       tw.i8_kv_attend_tree(c2, b2, q, m, max_len=max_len))
    path = dev(np.array([[0, 2, 3, 21, 25, 39]], np.int32))
    assert torch.equal(tw.i8_kv_keep(c, b, s.tokens, path), tw.i8_kv_keep(c2, b2, s.tokens, path))
    assert torch.equal(codes[far:], c.codes) and torch.equal(scales[far:], c.scales) and not codes[:far].any()


def test_blocks_that_are_not_there():
    s = Case(tw, 31, 64, 2, [40], [100])
    s.table[0, 1] = -1                                  # positions 64 to 127, rows 0 to 27
    check(s, queries(s, 4), forest(s.rng, [40]))
    s = Case(tw, 37, 64, 1, [20], [0])
    s.lens[0] = 12                                      # rows 0 to 7 in front of position 0
    got = check(s, queries(s, 2), forest(s.rng, [20]))
    assert np.all(got[:8] == 0)


def test_strided_queries_and_scale():
    import torch
    s = Case(tw, 41, 128, 2, [20], [333])
    q = queries(s, 4)
    rows = torch.zeros(20, 9, 128, dtype=torch.bfloat16, device="cuda")
    rows[:, 3:7] = dev(q, torch.bfloat16)
    c, b = s.device()
    m, _ = tw.draft_tree_mask(b, dev(grow(s.rng, 20)))
    assert torch.equal(tw.i8_kv_attend_tree(c, b, rows[:, 3:7], m, scale=-0.2),
                       tw.i8_kv_attend_tree(c, b, dev(q, torch.bfloat16), m, scale=-0.2))


# ---- accepted branch ----
@pytest.mark.parametrize("new, width", [([1], 1), ([64], 20), ([64], 3), ([5, 0, 17, 1], 8), ([512, 40], 600),
                                        ([700], 100)])
def test_accept(new, width):
    rng = np.random.default_rng([sum(new), width])
    for reach in (1, 3, 30):
        cu = np.concatenate([[0], np.cumsum(new)])
        parent = forest(rng, new, reach)
        token = rng.integers(0, 3, len(parent)).astype(np.int32)   # few tokens: siblings alike, long branches
        target = rng.integers(0, 3, len(parent)).astype(np.int32)
        got = tw.draft_tree_accept(batch_of(cu, np.full(len(new), 900)), dev(parent), dev(token), dev(target), width)
        for g, w in zip(got, tree.accept(cu, parent, token, target, width)):
            assert np.array_equal(host(g), w)


def test_accept_odd_input():
    rng = np.random.default_rng(9)
    parent = rng.integers(-40, 60, 90).astype(np.int32)
    token, target = rng.integers(0, 2, (2, 90)).astype(np.int32)
    for cu in ([0, 30, 60, 90], [0, 40, 20, 90], [0, 50, 95], [-3, 20, 60]):
        got = tw.draft_tree_accept(batch_of(cu, np.full(len(cu) - 1, 50)), dev(parent), dev(token), dev(target), 9)
        for g, w in zip(got, tree.accept(cu, parent, token, target, 9)):
            assert np.array_equal(host(g), w), cu


# ---- keep ----
def kept_cache(s, paths, table=None, lens_out=True):
    c = tw.I8KvCache(codes=dev(s.codes), scales=dev(s.scales))
    b = tw.I8KvBatch(dev(s.cu), dev(s.lens), dev(s.table if table is None else table))
    lens = host(tw.i8_kv_keep(c, b, s.tokens, dev(paths)))
    o = kv.Cache(s.codes, s.scales)
    want = tree.keep(o, s.cu, s.lens, s.table if table is None else table, s.tokens, paths)
    assert np.array_equal(lens, want)
    assert np.array_equal(host(c.scales), o.scales, equal_nan=True)
    got = host(c.codes)
    where = np.argwhere(got != o.codes)
    assert len(where) == 0, where[:5]


def ascending(rng, n, width, most=None):
    count = int(rng.integers(0, min(n, width if most is None else most) + 1))
    path = np.full(width, -1, np.int32)
    path[:count] = np.sort(rng.choice(n, count, replace=False))
    return path


@pytest.mark.parametrize("d, heads", [(128, 2), (64, 3)])
@pytest.mark.parametrize("new, prev", [([64], [30]), ([9], [60]), ([1, 40, 0, 64], [5, 0, 70, 63]), ([300], [10]),
                                       ([512, 17], [64, 64]), ([90], [127])])
def test_keep(d, heads, new, prev):
    for seed in range(3):
        s = Case(tw, [d, sum(new), seed], d, heads, new, prev)
        # scales far apart: some blocks must take tokens of much larger values
        s.scales *= np.exp2(s.rng.integers(-6, 7, s.scales.shape)).astype(np.float32)
        width = (8, 40, 600)[seed]
        kept_cache(s, np.stack([ascending(s.rng, n, width) for n in new]))


def test_keep_takes_what_ascends():
    s = Case(tw, 51, 64, 1, [64, 64, 64, 64, 600], [50, 50, 50, 50, 50])
    paths = np.full((5, 7), -1, np.int32)
    paths[0] = [0, 3, 3, 9, 20, 30, 40]
    paths[1] = [0, 3, 64, 9, 20, 30, 40]
    paths[2] = [5, 4, 9, 10, 20, 30, 40]
    paths[3] = np.arange(7)
    paths[4] = [0, 20, 400, 511, 512, 599, 5]
    kept_cache(s, paths)


def test_keep_special_scales():
    """Blocks of zeros, and scales that are not finite, as source and as place."""
    for a, b in ((0, 0.5), (0.5, 0), (0, 0), (np.inf, 0.5), (0.5, np.inf), (np.nan, 0.5), (0.5, np.nan), (0.5, 1e38),
                 (1e-38, 1e38), (np.inf, np.nan)):
        s = Case(tw, 53, 64, 2, [80], [40])
        s.scales[s.table[0, 0], 0], s.scales[s.table[0, 1], 0] = a, b
        kept_cache(s, np.array([[0, 5, 30, 50, 70, -1]], np.int32))


def test_keep_blocks_that_are_not_there():
    s = Case(tw, 57, 64, 2, [150], [40])
    path = np.array([[0, 5, 30, 50, 70, 100, 120, 140]], np.int32)
    for gone in (0, 1, 2):
        table = s.table.copy()
        table[0, gone] = (-1, 10 ** 6, -7)[gone]
        kept_cache(s, path, table)
    kept_cache(s, path, s.table[:, :2].copy())
    s.lens[0] = 100                                     # rows 0 to 49 in front of position 0
    kept_cache(s, np.concatenate([path, path + 3], 1)[:, [0, 1, 2, 3, 4, 5, 6, 7]])
    kept_cache(s, np.arange(0, 150, 2, dtype=np.int32)[None])


def test_keep_of_no_rows():
    import torch
    s = Case(tw, 59, 64, 1, [3, 0, 2], [10, 70, 0])
    c, b = s.device()
    before = host(c.codes)
    path = torch.zeros(3, 4, dtype=torch.int32, device="cuda") - 1
    assert host(tw.i8_kv_keep(c, b, s.tokens, path)).tolist() == [10, 70, 0]
    assert host(tw.i8_kv_keep(c, b, 0, path)).tolist() == [13, 70, 2]     # all rows outside
    descends = tw.I8KvBatch(dev(np.array([0, 3, 1, 5], np.int32)), b.lens, b.table)
    assert host(tw.i8_kv_keep(c, descends, s.tokens, path + 1)).tolist() == [11, 70, 2]
    assert np.array_equal(host(c.codes), before)


# ---- the step ----
def test_step_of_a_tree_is_a_step_of_its_branch():
    """Trees appended, attended, walked and cut to the accepted branch, through one captured graph, against the
    branches' tokens appended and attended one sequence at a time; then a next token over both caches."""
    import torch
    d, heads, hq, new, prev = 128, 2, 8, [40, 25, 1], [50, 700, 63]
    s = Case(tw, 61, d, heads, new, prev)
    f = tw.QkTransform(d, q_gain=dev(s.rng.uniform(0.5, 2, d).astype(np.float32)),
                       k_gain=dev(s.rng.uniform(0.5, 2, d).astype(np.float32)),
                       inv_freq=dev(1e6 ** (-np.arange(0, d, 2) / d)))
    c, b = s.device()
    start = c.codes.clone(), c.scales.clone()
    parent = forest(s.rng, new, 4)
    parent[s.cu[:-1]] = -1
    token = np.arange(s.tokens, dtype=np.int32)
    target = np.full(s.tokens, -5, np.int32)
    paths = []
    for i, n in enumerate(new):
        mine = parent[s.cu[i]:s.cu[i + 1]]
        best = max((tree.branch(mine, r)[::-1] for r in range(n) if tree.branch(mine, r)[-1] == 0), key=len)
        for x, y in zip(best, best[1:]):
            target[s.cu[i] + x] = token[s.cu[i] + y]
        paths.append(best)
    assert max(map(len, paths)) > 4
    rows = dev(s.rng.normal(size=(s.tokens, hq + 2 * heads, d)).astype(np.float32))
    q, k, v = rows[:, :hq], rows[:, hq:hq + heads], rows[:, hq + heads:]
    par, tok, tar = dev(parent), dev(token), dev(target)

    def step():
        mask, pos = tw.draft_tree_mask(b, par)
        qr = tw.i8_kv_append(c, b, f, k, v, q=q, pos=pos)
        out = tw.i8_kv_attend_tree(c, b, qr, mask)
        path, count, following = tw.draft_tree_accept(b, par, tok, tar, 40)
        return out, path, count, following, tw.i8_kv_keep(c, b, s.tokens, path)

    eager = step()
    after = c.codes.clone(), c.scales.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.codes.copy_(start[0]), c.scales.copy_(start[1])
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        c.codes.copy_(start[0]), c.scales.copy_(start[1])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, eager))
        assert torch.equal(c.codes, after[0]) and torch.equal(c.scales, after[1])
    assert host(eager[2]).tolist() == [len(p) for p in paths]
    assert host(eager[4]).tolist() == [p + len(x) for p, x in zip(prev, paths)]
    # the branches alone, in a cache of their own
    flat = np.concatenate([s.cu[i] + np.array(p) for i, p in enumerate(paths)])
    at = torch.from_numpy(flat).cuda()
    lone = tw.I8KvCache(codes=start[0].clone(), scales=start[1].clone())
    b2 = batch_of(np.concatenate([[0], np.cumsum([len(p) for p in paths])]), host(eager[4]), s.table)
    q2 = tw.i8_kv_append(lone, b2, f, k[at].contiguous(), v[at].contiguous(), q=q[at].contiguous())
    want = host(tw.i8_kv_attend(lone, b2, q2))
    got = host(eager[0][at])
    # both quantise keys and values to half a step of a block's scale, at most 2^-6 of its largest value once it
    # has grown; a score of size 4 or so moves by a few hundredths
    assert np.abs(got - want).max() <= 0.08 * np.abs(want).max()
    after_k, after_v = (host(x) for x in tw.i8_kv_read(c, b2, len(flat)))
    lone_k, lone_v = (host(x) for x in tw.i8_kv_read(lone, b2, len(flat)))
    top = np.maximum(host(c.scales).max(), host(lone.scales).max())
    assert np.abs(after_k - lone_k).max() <= 2 * top and np.abs(after_v - lone_v).max() <= 2 * top


def test_two_streams_at_once():
    """Trees of two batches on two streams, each with its own cache."""
    import torch
    parts = []
    for i in range(2):
        s = Case(tw, 71 + i, 128, 2, [30, 12], [4000, 900])
        c, b = s.device()
        m, _ = tw.draft_tree_mask(b, dev(forest(s.rng, [30, 12])))
        parts.append((c, b, dev(queries(s, 8), torch.bfloat16), m))
    want = [tw.i8_kv_attend_tree(*p) for p in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = [tw.i8_kv_attend_tree(*p, stream=st) for p, st in zip(parts, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_workspace_sized_for_the_largest_batch():
    """It serves smaller ones, which need one where the largest does not."""
    import torch
    s = Case(tw, 101, 64, 8, [24, 9, 24], [2000, 30, 700])
    c, b = s.device()
    lens = torch.zeros(140, dtype=torch.int32, device="cuda")
    many = tw.I8KvBatch(torch.zeros(141, dtype=torch.int32, device="cuda"), lens, b.table[:1].expand(140, -1).contiguous())
    assert tw.i8_kv_attend_tree_workspace_bytes(140 * 24, 32, 8, 64, 140, 16000) == 0
    ws = tw.i8_kv_attend_tree_workspace(c, many, 140 * 24, 32, 16000)
    m, _ = tw.draft_tree_mask(b, dev(forest(s.rng, [24, 9, 24])))
    q = dev(queries(s, 32), torch.bfloat16)
    for max_len in (None, 500, 16000, LONG):
        assert torch.equal(tw.i8_kv_attend_tree(c, b, q, m, max_len=max_len, workspace=ws),
                           tw.i8_kv_attend_tree(c, b, q, m, max_len=max_len))
