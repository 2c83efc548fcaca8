"""The prompt kernel of i8_kv_attend (256 columns a workgroup, fp16 matrix
cores) at its edges, against a 64-bit oracle: tiles whole, cut into stretches
and joined, and beside the launch for short sequences.  Every test asserts the
path it covers."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import kv

from test_gpu_kv import Case, dev, host, queries

pytestmark = pytest.mark.gpu

LONG = 10 ** 6                        # told of long caches, tiles are cut into stretches


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    assert torch.cuda.is_available()
    tw.lib()


def make(kind, seed, d=64, prev=500, rows=200):
    """A case of one kind of launch: (case, query heads, max_len)."""
    if kind == "split":
        return Case(tw, seed, d, 1, [rows], [prev]), 4, LONG
    if kind == "whole":
        return Case(tw, seed, d, 16, [600], [1500 if prev is None else max(prev, 1500)]), 64, None
    assert kind == "beside"
    return Case(tw, seed, d, 2, [1, rows, 3, 2], [max(prev, 700), prev, 60, 130]), 8, LONG


def path(s, hq, window, max_len):
    return tw.i8_kv_attend_config(s.tokens, hq, s.heads, s.d, len(s.lens), s.table.shape[1], window, max_len)


def assert_kind(kind, s, hq, window, max_len):
    launches = path(s, hq, window, max_len)
    assert launches[0]["cols"] == 256, launches
    assert len(launches) == (2 if kind == "beside" else 1) and (launches[0]["groups"] == 0) == (kind == "whole"), launches
    assert len(launches) == 1 or launches[1]["cols"] == 16


def attend(s, q, window=0, scale=None, max_len=None):
    import torch
    c, b = s.device()
    return host(tw.i8_kv_attend(c, b, dev(q, torch.bfloat16), scale=scale, window=window, max_len=max_len))


def exact(s, q, window=0, scale=None, rows=None):
    """(out, bound) fp64 [T, Hq, D], of all rows of all sequences or of the rows given.

    The bound, beside bf16's half step, of what the operands leave out.  With e
    the error of a score and A = sum w|v| / sum w, an output is off by 2 e A
    (numerator and denominator) and by what a weight in fp16 is off: 2^-11 A
    for its half step, and, where the weight's product with its block's scale
    falls below 2^-23 of the row's largest such product (held as 2^9 or more),
    half of fp16's smallest step, 2^-34 of that product, for each of n tokens
    of up to 127.  e is 2^-15 max|q| sum|k| scale (q in 15 bits, or to 2^-25 in
    fp16) and 2^-20 |score| of fp32 arithmetic.  The launch for short sequences
    has weights to 2^-16 of their block's largest: 64 * 2^-15 of max|v| there,
    which "short" rows are allowed in place of 2^-11 A.  In the
    tiles a smaller block scale than 2^-80 stands for that (2^-73 for codes of up
    to 127), and results below 2^-73 are 0: 2^-72 together."""
    scale = s.d ** -0.5 if scale is None else scale
    out = np.zeros(q.shape)
    bound = np.zeros(q.shape)
    cache = kv.Cache(s.codes, s.scales)
    g = q.shape[1] // s.heads
    for i in range(len(s.lens)):
        n, length = int(s.cu[i + 1] - s.cu[i]), max(int(s.lens[i]), 0)
        k, v, there = cache.sequence(s.table[i], length)
        sv = np.zeros((length, s.heads))
        for b in range(min(-(-length // 64), len(s.table[i]))):
            if 0 <= s.table[i, b] < len(s.codes):
                sv[b * 64:(b + 1) * 64] = s.scales[s.table[i, b], :, 1]
        js = np.arange(n)
        if rows is not None:
            js = js[np.isin(s.cu[i] + js, rows)]
        if len(js) == 0 or length == 0:
            continue
        p = length - n + js
        at = np.arange(length)
        seen = there & (at <= p[:, None])
        if window:
            seen &= at > p[:, None] - window
        for h in range(q.shape[1]):
            kk, vv = k[:, h // g], v[:, h // g]
            x = q[s.cu[i] + js, h].astype(np.float64)
            with np.errstate(invalid="ignore", over="ignore"):
                sc = np.where(seen, x @ kk.T * scale, -np.inf)
                top = np.where(seen.any(1), sc.max(1, initial=-np.inf), 0.0)[:, None]
                w = np.where(seen, np.exp(sc - top), 0.0)
                total = np.maximum(w.sum(1), 1e-300)[:, None]
                e = (2.0 ** -15 * np.abs(x).max(1) * np.where(seen, np.abs(kk).sum(1), 0).max(1) * abs(scale)
                     + 2.0 ** -20 * np.where(seen, np.abs(sc), 0).max(1))[:, None]
                o = w @ np.where(there[:, None], vv, 0) / total
                a = w @ np.abs(np.where(there[:, None], vv, 0)) / total
                most = (w * sv[:, h // g]).max(1, initial=0)[:, None] / total * 127
                short = n * g <= 128
                big = np.where(seen, np.abs(vv).max(1), 0).max(1)[:, None]
                part = 2.0 ** -9 * big if short else 2.0 ** -11 * a
                bound[s.cu[i] + js, h] = 2 * e * a + part + length * 2.0 ** -34 * most + 2.0 ** -72
                out[s.cu[i] + js, h] = o
    return out, bound


def check(kind, s, hq, q, window=0, scale=None, max_len=None):
    assert_kind(kind, s, hq, window, max_len)
    got = attend(s, q, window, scale, max_len)
    want, bound = exact(s, q, window, scale)
    err = np.abs(got - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + bound)
    return got


KINDS = ["split", "whole", "beside"]
PROMPT = {"split": 0, "whole": 0, "beside": 1}                  # which sequence


# ---- block scales of the values ----
@pytest.mark.parametrize("kind, d, k", [(kind, d, k) for kind in KINDS for d in (64, 128) for k in
                                        ((30, 100) if (kind, d) == ("whole", 128) else (20, 24, 30, 36, 60, 100))])
def test_larger_values_behind_a_row_do_not_reach_it(kind, d, k):
    """The last block's values are 2^k times the others': rows in front of it are as right as without it."""
    s, hq, max_len = make(kind, 200 + k, d)
    i = PROMPT[kind]
    s.scales[s.table[i, (s.lens[i] - 1) // 64], :, 1] *= np.float32(2.0) ** k
    check(kind, s, hq, queries(s, hq), max_len=max_len)


@pytest.mark.parametrize("k", [24, 36, 100])
def test_larger_values_in_front_of_a_window_do_not_reach_it(k):
    """Early blocks with values 2^k times the others', in front of the window of all but the first rows."""
    s = Case(tw, 300 + k, 64, 16, [600], [1500])
    s.scales[s.table[0, :3], :, 1] *= np.float32(2.0) ** k
    check("whole", s, 64, queries(s, 64), window=1750)


@pytest.mark.parametrize("k", [30, 60])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("kind", KINDS)
def test_larger_values_of_no_weight_do_not_drown_others(kind, first, k):
    """Blocks with values 2^k times the others' whose keys score 2 k below them: seen, and weighing nothing."""
    s, hq, max_len = make(kind, 310 + k)
    i = PROMPT[kind]
    q = np.ones((s.tokens, hq, 64), np.float32)
    blocks = s.table[i, :2] if first else s.table[i, (s.lens[i] - 1) // 64 - 1:][:1]
    s.codes[blocks, :, 0] = -100
    s.scales[blocks, :, 0] = 2 * k / 100 / 64 / 0.125
    s.scales[blocks, :, 1] *= np.float32(2.0) ** k
    check(kind, s, hq, q, max_len=max_len)


@pytest.mark.parametrize("kind", KINDS)
def test_uneven_scales(kind):
    """Blocks whose values differ by orders of magnitude, in no order, and blocks of zeros."""
    s, hq, max_len = make(kind, 320, 128, prev=900)
    i = PROMPT[kind]
    s.scales[:, :, 1] *= (10.0 ** s.rng.uniform(-9, 9, s.scales.shape[:2])).astype(np.float32)
    s.scales[s.table[i, 2]] = 0
    s.scales[s.table[i, 4], :, 1] = 0
    check(kind, s, hq, queries(s, hq), max_len=max_len)


@pytest.mark.parametrize("tiny", [0.0, 2.0 ** -140, 2.0 ** -110])
@pytest.mark.parametrize("kind", ["split", "whole"])
def test_rows_that_see_values_of_nothing(kind, tiny):
    """All blocks but the last have values of (nearly) nothing: rows in front of the last one give zeros
    (below 2^-73), and the others weigh those tokens as they should."""
    s, hq, max_len = make(kind, 330, prev=0 if kind == "split" else None)
    last = (s.lens[0] - 1) // 64
    s.scales[s.table[0, :last], :, 1] = tiny
    got = check(kind, s, hq, queries(s, hq), max_len=max_len)
    rows = int(last * 64 - (s.lens[0] - s.new[0]))
    assert rows > 0 and np.all(got[:rows] == 0) and np.all(np.abs(got[rows:]).max((1, 2)) > 0)


# ---- what a row sees ----
@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_see_nothing(kind):
    """Rows in front of the start give zeros, those behind them what they see; a sequence of length 0 gives
    zeros; rows of no sequence are left as they were."""
    import torch
    if kind == "whole":
        s, hq, max_len = Case(tw, 340, 64, 16, [600, 500], [1500, 0], spare_rows=3), 64, None
    else:
        s, hq, max_len = Case(tw, 340, 64, 2, [200, 170] + ([1, 0, 3] if kind == "beside" else []),
                              [500, 0] + ([300, 0, 60] if kind == "beside" else []), spare_rows=3), 8, LONG
    s.lens[:2] = s.new[0] - 77, 0
    if kind == "beside":
        s.lens[4] = 1
    tiles, short = path(s, hq, 0, max_len)
    assert (tiles["cols"], tiles["groups"] == 0, short["cols"]) == (256, kind == "whole", 16)
    q = queries(s, hq)
    c, b = s.device()
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    tw.i8_kv_attend(c, b, dev(q, torch.bfloat16), out=out, max_len=max_len)
    got, n = host(out), int(s.cu[-1])
    want, bound = exact(s, q)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[:n])
    assert np.all(got[:77] == 0) and np.all(np.abs(got[77:s.cu[1]]).max(-1) > 0)
    assert np.all(got[s.cu[1]:s.cu[2]] == 0) and np.all(got[n:] == 9)


@pytest.mark.parametrize("kind", KINDS)
def test_missing_blocks(kind):
    s, hq, max_len = make(kind, 350, prev=900)
    i = PROMPT[kind]
    s.table[i, [0, 3, 4, 5, 7, (s.lens[i] - 1) // 64]] = -1, 10 ** 6, -1, len(s.codes), -2 ** 31, -1
    check(kind, s, hq, queries(s, hq), max_len=max_len)
    s.table[i] = -1                                              # none at all: zeros
    got = check(kind, s, hq, queries(s, hq), max_len=max_len)
    assert np.all(got[s.cu[i]:s.cu[i + 1]] == 0)


@pytest.mark.parametrize("kind", KINDS)
def test_a_table_narrower_than_the_length(kind):
    """What the table does not hold is not seen; rows past it see all that it holds."""
    s, hq, max_len = make(kind, 355, prev=500)
    width = (int(s.lens[PROMPT[kind]]) - int(s.new[PROMPT[kind]]) + 100) // 64
    s.table = s.table[:, :width].copy()
    check(kind, s, hq, queries(s, hq), max_len=max_len or int(s.lens.max()))


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("kind", KINDS)
def test_scales_that_are_not_finite(kind, bad, side):
    """NaN in exactly the rows and heads that see the block, the others as without it."""
    s, hq, max_len = make(kind, 360, prev=700)
    i = PROMPT[kind]
    q = queries(s, hq)
    want, bound = exact(s, q)
    at = (int(s.lens[i]) - int(s.new[i])) // 64 + 2              # a block in the middle of the rows
    s.codes[s.table[i, at], -1, side] = 0
    s.scales[s.table[i, at], -1, side] = bad
    assert_kind(kind, s, hq, 0, max_len)
    got = attend(s, q, max_len=max_len)
    sees = np.zeros(got.shape[:2], bool)
    row = int(s.cu[i]) + at * 64 - (int(s.lens[i]) - int(s.new[i]))
    assert s.cu[i] < row < s.cu[i + 1]
    sees[row:s.cu[i + 1], hq - hq // s.heads:] = True
    assert np.array_equal(np.isnan(got), np.broadcast_to(sees[..., None], got.shape))
    ok = ~sees
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[ok])


@pytest.mark.parametrize("kind", KINDS)
def test_queries_that_are_not_finite(kind):
    s, hq, max_len = make(kind, 370)
    q = queries(s, hq)
    want, bound = exact(s, q)
    first = int(s.cu[PROMPT[kind]])
    places = [(first, 0, 3, np.nan), (first + 70, 1, 40, np.inf), (first + 131, hq - 1, 63, -np.inf)]
    for t, h, d, bad in places:
        q[t, h, d] = bad
    assert_kind(kind, s, hq, 0, max_len)
    got = attend(s, q, max_len=max_len)
    ok = np.ones(got.shape[:2], bool)
    for t, h, *_ in places:
        assert np.isnan(got[t, h]).all()
        ok[t, h] = False
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[ok])


@pytest.mark.parametrize("kind", KINDS)
def test_queries_of_any_size(kind):
    """Rows of zeros, of numbers too small to score, and of large ones (scores stay in range by the scale)."""
    s, hq, max_len = make(kind, 375)
    q = queries(s, hq)
    first = int(s.cu[PROMPT[kind]])
    q[first:first + 40] = 0
    q[first + 40:first + 80] *= np.float32(2.0) ** -110
    q[first + 80:first + 120] *= 2.0 ** -9
    q[first + 120:first + 130] *= 2.0 ** 5
    check(kind, s, hq, kv.bf16(q), max_len=max_len)


@pytest.mark.parametrize("kind", KINDS)
def test_what_is_masked_changes_nothing(kind):
    """Bytes behind the length, unused blocks and table entries behind the length."""
    s, hq, max_len = make(kind, 380)
    i = PROMPT[kind]
    s.table = np.concatenate([s.table, np.full((len(s.table), 2), 10 ** 9, np.int32)], 1)
    q = queries(s, hq)
    first = check(kind, s, hq, q, max_len=max_len or int(s.lens.max()))
    last, left = divmod(int(s.lens[i]) - 1, 64)
    assert left < 63
    for side in (0, 1):
        tail = kv.place(side, s.d)[left + 1:].ravel()
        s.codes[s.table[i, last], :, side][:, tail] = -127
    s.scales[np.setdiff1d(np.arange(len(s.codes)), s.table)] = np.nan
    assert np.array_equal(first, attend(s, q, max_len=max_len or int(s.lens.max())))


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.01, 0.3])
@pytest.mark.parametrize("kind", KINDS)
def test_scale(kind, scale):
    s, hq, max_len = make(kind, 390)
    check(kind, s, hq, queries(s, hq), scale=scale, max_len=max_len)


@pytest.mark.parametrize("rows", [130, 200])
def test_flat_tail(rows):
    """One key far above thousands of equal ones that together weigh as much."""
    s = Case(tw, 400, 64, 1, [rows], [6000])
    s.scales[:] = 0.01
    s.codes[:, :, 0] = 0
    s.codes[s.table[0, 0], 0, 0][kv.place(0, 64)[5]] = 100
    check("split", s, 4, np.ones((s.tokens, 4, 64), np.float32), scale=np.log(6000.0) / 64, max_len=LONG)


# ---- windows, and units of more blocks than a wave looks up at once ----
def sampled(s, q, window, max_len, step=37):
    rows = np.unique(np.concatenate([np.arange(0, s.tokens, step), [s.tokens - 1]]))
    got = attend(s, q, window, max_len=max_len)
    want, bound = exact(s, q, window, rows=rows)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[rows])
    return got


@pytest.mark.parametrize("new, prev, heads, hq, window, max_len, kind", [
    ([1000], [0], 8, 64, 70, None, "whole"), ([1000], [0], 16, 64, 200, None, "whole"),
    ([300], [1500], 16, 128, 1000, None, "whole"), ([2000], [4000], 4, 16, 5000, None, "whole"),
    ([300] * 70, [40 + i for i in range(70)], 1, 5, 333, LONG, "whole"),
    ([400, 1, 3, 2], [4500, 300, 60, 0], 16, 64, 3000, LONG, "split"),
])
def test_windows(new, prev, heads, hq, window, max_len, kind):
    s = Case(tw, 410, 64, heads, new, prev)
    launches = path(s, hq, window, max_len)
    assert (launches[0]["cols"], launches[0]["groups"] == 0) == (256, kind == "whole")
    sampled(s, queries(s, hq), window, max_len)


@pytest.mark.parametrize("side", [0, 1])
def test_what_lies_in_front_of_a_window_changes_nothing(side):
    """Scales that are not finite: NaN in the rows whose window still holds the block, the others as without."""
    s = Case(tw, 420, 64, 8, [1000], [0])
    q = queries(s, 64)
    assert_kind("whole", s, 64, 70, None)
    want, bound = exact(s, q, 70)
    s.scales[s.table[0, [2, 6]], :, side] = np.nan
    got = attend(s, q, 70)
    p = np.arange(1000)
    sees = np.zeros(1000, bool)
    for b in (2, 6):
        sees |= (p >= 64 * b) & (p - 70 + 1 <= 64 * b + 63)
    assert np.array_equal(np.isnan(got).all((1, 2)), sees) and np.array_equal(np.isnan(got).any((1, 2)), sees)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[~sees])


@pytest.mark.parametrize("kind, new, prev, heads, hq, max_len", [
    ("whole", 600, 4200, 8, 64, None), ("split", 2000, 3000, 8, 32, LONG),
])
def test_units_of_many_blocks(kind, new, prev, heads, hq, max_len):
    """Uneven scales and missing blocks on both sides of the 64 blocks that are looked up together."""
    s = Case(tw, 430, 64, heads, [new], [prev])
    s.scales[:, :, 1] *= (2.0 ** s.rng.integers(-20, 20, s.scales.shape[:2])).astype(np.float32)
    s.table[0, [1, 62, 63, 64, 70]] = -1
    s.scales[s.table[0, 65]] = 0
    assert_kind(kind, s, hq, 0, max_len)
    tiles, most = -(-new * hq // heads // 256), -(-(new + prev) // 64)
    assert most > 64 and (kind == "whole" or tiles * heads * most > 64 * 256)        # of a unit, of a stretch
    sampled(s, queries(s, hq), 0, max_len)


# ---- calls ----
@pytest.mark.parametrize("kind", KINDS)
def test_equal_bytes_on_any_stream(kind):
    import torch
    s, hq, max_len = make(kind, 440, 128)
    assert_kind(kind, s, hq, 0, max_len)
    c, b = s.device()
    q = dev(queries(s, hq), torch.bfloat16)
    first = tw.i8_kv_attend(c, b, q, max_len=max_len)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = [tw.i8_kv_attend(c, b, q, max_len=max_len, stream=x) for x in (side, None, side)]
        torch.cuda.synchronize()
        assert all(torch.equal(first, x) for x in got)


def test_one_workspace_through_calls_and_graphs():
    import torch
    parts = []
    for i, kind in enumerate(KINDS):
        s, hq, max_len = make(kind, 450 + i)
        assert_kind(kind, s, hq, 0, max_len)
        parts.append((*s.device(), dev(queries(s, hq), torch.bfloat16), max_len))
    alone = [tw.i8_kv_attend(c, b, q, max_len=n) for c, b, q, n in parts]
    sizes = [tw.i8_kv_attend_workspace(c, b, len(q), q.shape[1], n) for c, b, q, n in parts]
    ws = torch.full((max(w.numel() for w in sizes if w is not None),), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(a) for a in alone]
    graphs = []
    for (c, b, q, n), out in zip(parts, outs):
        tw.i8_kv_attend(c, b, q, max_len=n, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tw.i8_kv_attend(c, b, q, max_len=n, out=out, workspace=ws)
        graphs.append(g)
    for order in ((0, 1, 2), (2, 0, 1), (1, 1, 0)):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], alone[i])
            c, b, q, n = parts[i]
            assert torch.equal(tw.i8_kv_attend(c, b, q, max_len=n, workspace=ws), alone[i])


def test_far_blocks_of_a_large_cache():
    """Blocks whose bytes lie past 2^32."""
    import torch
    d, heads, hq, rows = 128, 8, 16, 250
    blocks = 2 ** 32 // (heads * 2 * 64 * d) + 40
    codes = torch.zeros((blocks, heads, 2, 64 * d), dtype=torch.int8, device="cuda")
    far = tw.I8KvCache(codes=codes, scales=torch.zeros((blocks, heads, 2), device="cuda"))
    near = tw.I8KvCache(4, heads, d)
    rng = np.random.default_rng(460)
    k, v = dev(rng.normal(size=(2, rows, heads, d)).astype(np.float32))
    q = dev(rng.normal(size=(rows, hq, d)), torch.bfloat16)
    cu, lens = dev(np.array([0, rows], np.int32)), dev(np.array([rows], np.int32))
    assert tw.i8_kv_attend_config(rows, hq, heads, d, 1, 4, max_len=LONG)[0]["cols"] == 256
    got = []
    for cache, table in ((far, [blocks - 1, 3, blocks - 7, blocks // 2]), (near, [0, 1, 2, 3])):
        b = tw.I8KvBatch(cu, lens, torch.tensor([table], dtype=torch.int32, device="cuda"))
        tw.i8_kv_append(cache, b, tw.QkTransform(d), k, v)
        got.append(tw.i8_kv_attend(cache, b, q, max_len=LONG))
    assert torch.equal(*got)
