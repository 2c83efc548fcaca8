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
@pytest.mark.parametrize("k", [20, 24, 30, 36, 60, 100])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_larger_values_behind_a_row_do_not_reach_it(kind, d, k):
    """The last block's values are 2^k times the others': rows in front of it are as right as without it."""
    if d == 128 and kind == "whole" and k not in (30, 100):
        pytest.skip("two of six are enough at this size")
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
