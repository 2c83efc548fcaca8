"""The attention side of a decode step on the GPU against the 64-bit oracle
(oracle/kv.py): norm with rotation, the paged int8 cache's append and read,
attention over it, and the step they make together with the linears."""
import numpy as np
import pytest

import oracle
from oracle import kv
from ternary_weight_decode_amd import synth

pytestmark = pytest.mark.gpu

F = lambda d: 1e6 ** (-np.arange(0, d, 2) / d)


@pytest.fixture(scope="module")
def tw():
    import torch
    import ternary_weight_decode_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    import torch
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# ---- norm + rotation ----
# Tolerance.  The norm's sum of 64 or 128 squares, division and root come to
# at most 12 * 2^-24 relative, cos and sin to 5.2 * 2^-24 (the angle's fp32
# rounding, pi * 2^-24, and two units of sincospi), the two products and their
# sum to 3 * 2^-24: together 21 * 2^-24 of |a| + |b| for the pair (a, b);
# 2^-19 is allowed, and bf16 outputs add half a step, 2^-8 of the value.
def pair_size(x, interleaved):
    d = x.shape[-1]
    a = np.abs(x)
    if interleaved:
        s = a[..., 0::2] + a[..., 1::2]
        return np.repeat(s, 2, -1)
    s = a[..., :d // 2] + a[..., d // 2:]
    return np.concatenate([s, s], -1)


@pytest.mark.parametrize("d, hq, hk, tokens, interleaved, in16, out16, gain, freq", [
    (128, 32, 8, 1, False, False, True, True, True),
    (128, 16, 8, 5, False, False, False, True, True),
    (128, 3, 1, 67, True, False, False, True, True),
    (64, 7, 7, 33, False, True, True, True, True),
    (64, 1, 0, 2, True, True, False, True, True),
    (64, 0, 5, 130, True, False, True, True, True),
    (128, 4, 2, 9, False, True, False, False, True),
    (128, 4, 2, 9, False, False, False, True, False),
    (64, 17, 3, 4, False, True, True, False, False),
])
def test_norm_rope(tw, d, hq, hk, tokens, interleaved, in16, out16, gain, freq):
    import torch
    rng = np.random.default_rng([d, hq, hk, tokens])
    rows = (rng.normal(size=(tokens, hq + 2 * hk + 1, d)) * np.exp(rng.normal(size=(tokens, hq + 2 * hk + 1, 1))))
    rows = rows.astype(np.float32)
    if in16:
        rows = kv.bf16(rows)
    qg, kg = rng.uniform(0.3, 2, (2, d)).astype(np.float32)
    pos = rng.integers(0, 2 ** 20, tokens).astype(np.int32)
    pos[0], pos[-1] = 0, 2 ** 24
    f = tw.QkTransform(d, dev(qg) if gain else None, dev(kg) if gain else None, 1e-6, dev(F(d)) if freq else None,
                       interleaved)
    x = dev(rows, torch.bfloat16 if in16 else torch.float32)
    q = x[:, :hq] if hq else None
    k = x[:, hq:hq + hk] if hk else None
    got = tw.qk_norm_rope(f, q, k, dev(pos) if freq else None, out_dtype=torch.bfloat16 if out16 else torch.float32)
    for y, lo, n, g in ((got[0], 0, hq, qg), (got[1], hq, hk, kg)):
        if n == 0:
            assert y is None
            continue
        want = kv.transform(rows[:, lo:lo + n], g if gain else None, 1e-6, F(d) if freq else None, interleaved, pos)
        before = kv.transform(rows[:, lo:lo + n], g if gain else None, 1e-6, None, interleaved, pos)
        tol = 2.0 ** -19 * pair_size(before, interleaved) + (2.0 ** -8 * np.abs(want) if out16 else 0)
        assert np.all(np.abs(host(y) - want) <= tol)


def test_norm_rope_writes_its_rows_only(tw):
    import torch
    f = tw.QkTransform(64)
    x = dev(np.arange(4 * 3 * 64, dtype=np.float32).reshape(4, 3, 64))
    out = torch.full((6, 3, 64), 7.0, device="cuda")
    tw.qk_norm_rope(f, x[1:3], None, q_out=out[2:4])
    got = host(out)
    assert np.array_equal(got[2:4], host(x)[1:3]) and np.all(got[:2] == 7) and np.all(got[4:] == 7)


# ---- cache ----
def pages(rng, lens, width=None, spare=3):
    """A table of distinct shuffled blocks for sequences of these lengths; -1 where there is none."""
    need = [-(-max(n, 0) // 64) for n in lens]
    width = width or max(1, max(need))
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def filled(rng, blocks, heads, d):
    """A cache whose every slot holds something."""
    codes = rng.integers(-127, 128, (blocks, heads, 2, 64 * d)).astype(np.int8)
    scales = rng.uniform(0.01, 0.04, (blocks, heads, 2)).astype(np.float32)
    return codes, scales


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


class Case:
    def __init__(self, tw, seed, d, heads, new, prev, spare_rows=0):
        self.rng = np.random.default_rng(seed)
        self.new, self.prev = np.array(new), np.array(prev)
        self.cu, self.lens = offsets(new), (self.new + self.prev).astype(np.int32)
        self.table, blocks = pages(self.rng, self.lens)
        self.codes, self.scales = filled(self.rng, blocks, heads, d)
        self.tokens = int(self.cu[-1]) + spare_rows
        self.d, self.heads = d, heads
        self.tw = tw

    def device(self):
        c = self.tw.I8KvCache(codes=dev(self.codes), scales=dev(self.scales))
        b = self.tw.I8KvBatch(dev(self.cu), dev(self.lens), dev(self.table))
        return c, b


SEQS = [
    ([1], [0]), ([1], [63]), ([1], [64]), ([7], [60]), ([64], [0]), ([65], [1]), ([200], [0]),
    ([1, 1, 1], [0, 100, 63]), ([3, 0, 130, 1], [62, 70, 0, 640]), ([1] * 70, list(range(0, 210, 3))),
]


@pytest.mark.parametrize("new, prev", SEQS)
@pytest.mark.parametrize("d, heads, in16", [(128, 2, False), (64, 3, True)])
def test_append_bytes_without_transform(tw, new, prev, d, heads, in16):
    """No norm and no rotation: codes and scales byte for byte, old slots requantised where the new
    values are larger, everything else as it was."""
    import torch
    s = Case(tw, 5 + len(new) + prev[0], d, heads, new, prev, spare_rows=2)
    k, v = (s.rng.normal(size=(2, s.tokens, heads, d)) * 4.0 ** s.rng.integers(-2, 3, (2, s.tokens, heads, 1)))
    k, v = k.astype(np.float32), v.astype(np.float32)
    if in16:
        k, v = kv.bf16(k), kv.bf16(v)
    t16 = torch.bfloat16 if in16 else torch.float32
    c, b = s.device()
    assert tw.i8_kv_append(c, b, tw.QkTransform(d), dev(k, t16), dev(v, t16)) is None
    want = kv.Cache(s.codes, s.scales)
    want.append(s.cu, s.lens, s.table, k, v)
    assert np.array_equal(host(c.scales).view(np.uint32), want.scales.view(np.uint32))
    assert np.array_equal(host(c.codes), want.codes)


@pytest.mark.parametrize("new, prev", SEQS)
@pytest.mark.parametrize("d, heads, group, interleaved, own_pos", [(128, 2, 4, False, False), (64, 1, 3, True, True)])
def test_append_with_transform(tw, new, prev, d, heads, group, interleaved, own_pos):
    """Norm and rotation on the way: every new key within half a step (and the 2^-19 of its pair that
    the fp32 arithmetic may cost) of its exact value; q as qk_norm_rope gives it, bit for bit; rows
    behind the last sequence untouched."""
    import torch
    s = Case(tw, 11 + len(new) + prev[0], d, heads, new, prev, spare_rows=3)
    rows = s.rng.normal(size=(s.tokens, heads * (group + 2), d)).astype(np.float32)
    qg, kg = s.rng.uniform(0.3, 2, (2, d)).astype(np.float32)
    f = tw.QkTransform(d, dev(qg), dev(kg), 1e-6, dev(F(d)), interleaved)
    place = np.zeros(s.tokens, np.int32)
    for i in range(len(new)):
        place[s.cu[i]:s.cu[i + 1]] = s.prev[i] + np.arange(new[i])
    if own_pos:
        place = s.rng.integers(0, 10 ** 6, s.tokens).astype(np.int32)
    x = dev(rows)
    hq = heads * group
    q, k, v = x[:, :hq], x[:, hq:hq + heads], x[:, hq + heads:]
    c, b = s.device()
    q_out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    tw.i8_kv_append(c, b, f, k, v, q=q, pos=dev(place) if own_pos else None, q_out=q_out)
    alone = tw.qk_norm_rope(f, q, k, dev(place))[0]
    n = int(s.cu[-1])
    assert np.array_equal(host(q_out[:n]), host(alone[:n])) and np.all(host(q_out[n:]) == 5)
    before = kv.transform(rows[:, hq:hq + heads], kg, 1e-6, None, interleaved, place)
    exact = kv.transform(rows[:, hq:hq + heads], kg, 1e-6, F(d), interleaved, place)
    kr, vr = tw.i8_kv_read(c, b, s.tokens, dtype=torch.float32)
    scales = host(c.scales)
    got = host(kr)
    slack = 2.0 ** -19 * pair_size(before, interleaved)
    for i in range(len(new)):
        for j in range(new[i]):
            step = scales[s.table[i, (s.prev[i] + j) // 64], :, 0][:, None]
            row = s.cu[i] + j
            # half a step, the step itself rounded to fp32 (2^-24 of the value) and the product's rounding
            tol = step * 0.5 * (1 + 2.0 ** -16) + slack[row] + 2.0 ** -22 * np.abs(exact[row])
            assert np.all(np.abs(got[row] - exact[row]) <= tol)
    want = kv.Cache(s.codes, s.scales)              # v has no transform: its side byte for byte
    want.append(s.cu, s.lens, s.table, exact.astype(np.float32), host(v))
    assert np.array_equal(host(c.codes)[:, :, 1], want.codes[:, :, 1])


def test_append_special_values(tw):
    """Zeros, tiny values, an infinity, a NaN; a block started anew forgets them."""
    s = Case(tw, 3, 64, 1, [2] * 5, [62, 62, 62, 62, 0])
    k = s.rng.normal(size=(10, 1, 64)).astype(np.float32)
    k[0:2] = 0
    k[2:4] = 1e-42
    k[5, 0, 7] = np.inf
    k[6, 0, 9] = np.nan
    s.scales[s.table[0, 0]] = 0
    s.scales[s.table[4, 0]] = np.nan
    v = -k[::-1].copy()
    c, b = s.device()
    tw.i8_kv_append(c, b, tw.QkTransform(64), dev(k), dev(v))
    want = kv.Cache(s.codes, s.scales)
    want.append(s.cu, s.lens, s.table, k, v)
    assert np.array_equal(host(c.scales), want.scales, equal_nan=True)
    assert np.array_equal(host(c.codes), want.codes)
    assert np.isnan(want.scales).any() and np.isinf(want.scales).any()
    # a growing block whose old scale is not finite keeps it
    tw.i8_kv_append(c, tw.I8KvBatch(dev(s.cu), dev(s.lens), dev(s.table)), tw.QkTransform(64), dev(k * 0 + 1),
                    dev(v * 0 + 1))
    want.append(s.cu, s.lens, s.table, k * 0 + 1, v * 0 + 1)
    assert np.array_equal(host(c.scales), want.scales, equal_nan=True)


def test_append_and_read_skip_what_is_not_there(tw):
    """Positions below 0 and past the table, entries outside the cache, sequences whose rows descend
    or leave the tensor: nothing stored, zeros read, q still written for rows of a sequence."""
    import torch
    d, heads = 64, 2
    rng = np.random.default_rng(8)
    cu = np.array([0, 4, 8, 12, 10, 10, 40], np.int32)
    lens = np.array([2, 130, 66, 64, 64, 64], np.int32)         # 2 < 4 rows; 130 past 2 blocks
    table = np.array([[0, 1], [2, 3], [5, 99], [6, 7], [8, 9], [10, 11]], np.int32)
    table[1, 1] = -3
    codes, scales = filled(rng, 12, heads, d)
    k, v = rng.normal(size=(2, 14, heads, d)).astype(np.float32)
    c = tw.I8KvCache(codes=dev(codes), scales=dev(scales))
    b = tw.I8KvBatch(dev(cu), dev(lens), dev(table))
    q_out = torch.full((14, heads, d), 5.0, dtype=torch.bfloat16, device="cuda")
    tw.i8_kv_append(c, b, tw.QkTransform(d), dev(k), dev(v), q=dev(k), q_out=q_out)
    want = kv.Cache(codes, scales)
    good = [0, 1, 2]
    for i in good:
        n = cu[i + 1] - cu[i]
        want.append([0, n], lens[i:i + 1], table[i:i + 1], k[cu[i]:cu[i + 1]], v[cu[i]:cu[i + 1]])
    assert np.array_equal(host(c.scales), want.scales) and np.array_equal(host(c.codes), want.codes)
    assert np.array_equal(host(q_out[:12]), kv.bf16(k[:12])) and np.all(host(q_out[12:]) == 5)
    kr = torch.full((14, heads, d), 3.0, device="cuda")
    vr = torch.full((14, heads, d), 3.0, device="cuda")
    tw.i8_kv_read(c, b, 14, k_out=kr, v_out=vr)
    for i in good:
        ko, vo = want.read([0, cu[i + 1] - cu[i]], lens[i:i + 1], table[i:i + 1], cu[i + 1] - cu[i])
        assert np.array_equal(host(kr)[cu[i]:cu[i + 1]], ko.astype(np.float32))
        assert np.array_equal(host(vr)[cu[i]:cu[i + 1]], vo.astype(np.float32))
    assert np.all(host(kr)[12:] == 3) and np.all(host(vr)[12:] == 3)


@pytest.mark.parametrize("d, heads", [(128, 2), (64, 1)])
@pytest.mark.parametrize("new, prev", SEQS)
def test_read(tw, d, heads, new, prev):
    """fp32: code * scale, one rounding; bf16 the same rounded once more to the nearest."""
    import torch
    s = Case(tw, 21, d, heads, new, prev)
    c, b = s.device()
    want = kv.Cache(s.codes, s.scales).read(s.cu, s.lens, s.table, s.tokens)
    for got, w in zip(tw.i8_kv_read(c, b, s.tokens, dtype=torch.float32), want):
        assert np.array_equal(host(got), w.astype(np.float32))
    for got, w in zip(tw.i8_kv_read(c, b, s.tokens), want):
        assert np.array_equal(host(got), kv.bf16(w.astype(np.float32)))


# ---- attention ----
def check_attend(tw, s, q, window=0, scale=None, max_len=None, max_rows=0):
    """Within half a bf16 step of the exact value and the oracle's bound for the narrower operands;
    bf16's rounding alone is at most 2^-8 / sqrt(3) = 2^-8.79 of the value in the mean, so the root mean
    square of all errors is asked to stay below 2^-8 of the output's."""
    import torch
    c, b = s.device()
    got = host(tw.i8_kv_attend(c, b, dev(q, torch.bfloat16), scale=scale, window=window, max_len=max_len,
                               max_rows=max_rows))
    want, bound = kv.attend(kv.Cache(s.codes, s.scales), s.cu, s.lens, s.table, q,
                            s.d ** -0.5 if scale is None else scale, window)
    rows = slice(0, int(s.cu[-1]))
    err = np.abs(got - want)[rows]
    assert np.all(err <= (2.0 ** -8 * np.abs(want) + bound)[rows])
    assert np.sqrt((err ** 2).mean()) <= 2.0 ** -8 * np.sqrt((want[rows] ** 2).mean())
    return got


def queries(s, hq, size=1.5):
    return kv.bf16(s.rng.normal(size=(s.tokens, hq, s.d)) * size)


@pytest.mark.parametrize("d, heads, hq", [(128, 2, 8), (64, 2, 4), (128, 1, 1), (64, 1, 3), (128, 1, 20)])
@pytest.mark.parametrize("new, prev", [
    ([1], [0]), ([1], [63]), ([1], [64]), ([1], [1000]), ([7], [380]), ([16], [130]), ([64], [0]), ([97], [45]),
    ([150, 33], [0, 300]), ([1, 1, 1], [0, 517, 63]), ([1, 2, 0, 5, 1], [700, 62, 9, 0, 64]),
])
def test_attend(tw, d, heads, hq, new, prev):
    s = Case(tw, 31 + len(new) + prev[0], d, heads, new, prev)
    check_attend(tw, s, queries(s, hq))


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200])
@pytest.mark.parametrize("new, prev", [([1], [500]), ([5, 1], [190, 3]), ([140], [77])])
def test_attend_window(tw, new, prev, window):
    s = Case(tw, 41 + window, 128, 2, new, prev)
    check_attend(tw, s, queries(s, 8), window=window)


@pytest.mark.parametrize("new, prev, window", [
    ([1], [3900], 2871), ([1, 1], [100, 5000], 2500), ([6], [3900], 2500), ([20, 20, 3], [3000, 10, 2600], 2600),
    ([300], [4000], 3100), ([280, 1, 260], [3500, 4000, 10], 3333),
])
@pytest.mark.parametrize("max_len", [None, 10 ** 6])
def test_attend_long_window(tw, new, prev, window, max_len):
    """Windows long enough to be split."""
    s = Case(tw, 61, 64, 1, new, prev)
    check_attend(tw, s, queries(s, 4), window, max_len=max_len)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.01, 0.3])
@pytest.mark.parametrize("new, prev", [([1], [300]), ([90], [40])])
def test_attend_scale(tw, new, prev, scale):
    s = Case(tw, 47, 64, 1, new, prev)
    check_attend(tw, s, queries(s, 4), scale=scale)


@pytest.mark.parametrize("new", [1, 6, 40])
def test_attend_many_sequences_and_lengths(tw, new):
    s = Case(tw, 51 + new, 64, 2, [new] * 67, [(i * 37) % 300 for i in range(67)])
    check_attend(tw, s, queries(s, 4))


@pytest.mark.parametrize("new, max_len", [(1, None), (1, 64), (1, 10 ** 6), (16, 1), (60, None), (60, 128)])
def test_attend_long(tw, new, max_len):
    """Long enough to be split; max_len is a hint, right or wrong."""
    s = Case(tw, 53, 128, 1, [new, new], [9001, 1200])
    check_attend(tw, s, queries(s, 4), max_len=max_len)


@pytest.mark.parametrize("new, prev", [
    ([700], [0]), ([256], [900]), ([257], [63]), ([600], [1500]), ([300, 257, 513], [100, 0, 700]),
    ([300] * 70, [40] * 70), ([1200], [5]),
])
@pytest.mark.parametrize("d, heads, hq, window", [(64, 2, 6, 0), (128, 1, 1, 0), (128, 1, 8, 0), (64, 1, 5, 333)])
def test_attend_prompts_split_where_a_stretch_ends(tw, new, prev, d, heads, hq, window):
    # told of long caches, the tiles of all prompts are cut into equal stretches
    s = Case(tw, 131, d, heads, new, prev)
    check_attend(tw, s, queries(s, hq), window, max_len=10 ** 6)


@pytest.mark.parametrize("new, prev, heads, hq, max_len", [
    ([5] * 6, [200, 0, 64, 700, 3, 130], 2, 8, 10 ** 6), ([12, 0, 12, 9], [300, 5, 1000, 55], 2, 8, 10 ** 6),   # split
    ([10] * 80, [3 * i for i in range(80)], 32, 64, None), ([20] * 80, [3 * i for i in range(80)], 32, 64, None),
    ([7, 0, 20, 1] * 20, [5 * i for i in range(80)], 32, 64, None),                 # two and four tiles a workgroup
    ([300] * 40, [7] * 40, 8, 8, 10 ** 6), ([300, 1, 0, 2] * 30, list(range(120)), 8, 8, 10 ** 6),  # many 256-column tiles
])
def test_attend_batches_of_many_tiles(tw, new, prev, heads, hq, max_len):
    s = Case(tw, 137, 64, heads, new, prev)
    check_attend(tw, s, queries(s, hq), max_len=max_len)


@pytest.mark.parametrize("seqs, rows", [(70, 1), (130, 1), (70, 5)])
def test_attend_many_long_sequences(tw, seqs, rows):
    """More sequences than lanes, long enough to be split, some without rows."""
    s = Case(tw, 113 + seqs, 64, 1, [rows if i % 7 else 0 for i in range(seqs)], [(i * 311) % 2500 for i in range(seqs)])
    check_attend(tw, s, queries(s, 2))


@pytest.mark.parametrize("new", [1, 5, 150])
def test_rows_in_front_of_the_first_sequence(tw, new):
    """cu need not start at 0: rows in front of cu[0] are neither read nor written."""
    import torch
    s = Case(tw, 127, 64, 2, [new, new], [1200, 3])
    q = queries(s, 4)
    c, b = s.device()
    want = host(tw.i8_kv_attend(c, b, dev(q, torch.bfloat16)))
    late = tw.I8KvBatch(b.cu + 3, b.lens, b.table)
    pad = torch.full((3, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = torch.full((s.tokens + 3, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    tw.i8_kv_attend(c, late, torch.cat([pad, dev(q, torch.bfloat16)]), out=out)
    assert np.array_equal(host(out[3:]), want) and np.all(host(out[:3]) == 9)
    k = dev(s.rng.normal(size=(s.tokens, 2, 64)).astype(np.float32))
    other = tw.I8KvCache(codes=c.codes.clone(), scales=c.scales.clone())
    tw.i8_kv_append(c, b, tw.QkTransform(64), k, k)
    tw.i8_kv_append(other, late, tw.QkTransform(64), torch.cat([pad[:, :2].float(), k]),
                    torch.cat([pad[:, :2].float(), k]))
    assert torch.equal(c.codes, other.codes) and torch.equal(c.scales, other.scales)


def test_one_workspace_for_calls_in_turn(tw):
    """A workspace carries nothing from call to call: different batches through one, and through graphs
    that share it, give what they give alone."""
    import torch
    cases = [Case(tw, 131 + i, 128, 2, new, prev) for i, (new, prev) in
             enumerate([([1], [5000]), ([1, 3, 200], [3000, 10, 1500]), ([12], [2000]), ([400], [900])])]
    parts = [(*s.device(), dev(queries(s, 8), torch.bfloat16)) for s in cases]
    alone = [tw.i8_kv_attend(*p) for p in parts]
    sizes = [tw.i8_kv_attend_workspace(c, b, len(q), 8) for c, b, q in parts]
    ws = torch.full((max(w.numel() for w in sizes if w is not None),), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(a) for a in alone]
    graphs = []
    for (c, b, q), out in zip(parts, outs):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            tw.i8_kv_attend(c, b, q, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tw.i8_kv_attend(c, b, q, out=out, workspace=ws)
        graphs.append(g)
    for order in ((0, 1, 2, 3), (3, 1, 0, 2), (2, 2, 1, 0)):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], alone[i])
            assert torch.equal(tw.i8_kv_attend(*parts[i], workspace=ws), alone[i])


def test_calls_overlap_on_two_streams(tw):
    """Appends to two caches and attention over them, on two streams at once."""
    import torch
    s = [Case(tw, 137 + i, 128, 2, [33, 1], [1000, 40 + i]) for i in range(2)]
    parts = [x.device() for x in s]
    k = [dev(x.rng.normal(size=(x.tokens, 2, 128)).astype(np.float32)) for x in s]
    q = [dev(queries(x, 8), torch.bfloat16) for x in s]
    f = tw.QkTransform(128)
    want = []
    for i in range(2):
        c = tw.I8KvCache(codes=parts[i][0].codes.clone(), scales=parts[i][0].scales.clone())
        tw.i8_kv_append(c, parts[i][1], f, k[i], k[i])
        want.append(tw.i8_kv_attend(c, parts[i][1], q[i]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for i in range(2):
            tw.i8_kv_append(*parts[i], f, k[i], k[i], stream=streams[i])
            got.append(tw.i8_kv_attend(*parts[i], q[i], stream=streams[i]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("new, prev, max_rows", [
    ([200, 1, 1, 150, 3, 0, 32, 33], [900, 2000, 5, 0, 1300, 3, 700, 40], 0),      # both paths, either side of 128 columns
    ([1, 1, 400], [3000, 70, 1200], 0), ([1, 1, 400], [3000, 70, 1200], 400), ([1, 1, 400], [3000, 70, 1200], 1),
    ([300, 300], [1200, 64], 0), ([2] * 20 + [140], [1500] * 20 + [2], 140),
])
@pytest.mark.parametrize("d, heads, hq, window", [(128, 8, 32, 0), (64, 4, 16, 500)])
def test_attend_prompts_beside_single_tokens(tw, new, prev, max_rows, d, heads, hq, window):
    s = Case(tw, 109 + len(new), d, heads, new, prev)
    check_attend(tw, s, queries(s, hq), window=window, max_rows=max_rows)


@pytest.mark.parametrize("new", [1, 3, 50])
def test_attend_flat_tail(tw, new):
    """One key far above thousands of equal ones that together weigh as much: none of them may vanish."""
    s = Case(tw, 57, 64, 1, [new], [6000])
    place = kv.place(0, 64)
    s.scales[:] = 0.01
    s.codes[:, :, 0] = 0
    s.codes[s.table[0, 0], 0, 0][place[5]] = 100
    q = np.ones((s.tokens, 2, 64), np.float32)
    check_attend(tw, s, q, scale=np.log(6000.0) / 64)


@pytest.mark.parametrize("new", [1, 4, 70])
def test_attend_uneven_scales(tw, new):
    """Blocks whose values differ by orders of magnitude, and blocks of zeros."""
    s = Case(tw, 59, 128, 1, [new], [900])
    s.scales[:, :, 1] *= (10.0 ** s.rng.uniform(-3, 3, s.scales.shape[:2])).astype(np.float32)
    s.scales[s.table[0, 2]] = 0
    s.scales[s.table[0, 4], :, 1] = 0
    check_attend(tw, s, queries(s, 4))


@pytest.mark.parametrize("new", [1, 5, 80])
def test_attend_rows_that_see_nothing(tw, new):
    """Rows in front of the start and sequences of length 0 give zeros; rows behind the last sequence
    are left as they were."""
    import torch
    s = Case(tw, 61, 64, 2, [new, new, new], [200, 0, 10], spare_rows=2)
    s.lens = np.array([200 + new, new - new // 2 - 1, 0], np.int32)
    q = queries(s, 4)
    c, b = s.device()
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    tw.i8_kv_attend(c, b, dev(q, torch.bfloat16), out=out)
    got = host(out)
    want, bound = kv.attend(kv.Cache(s.codes, s.scales), s.cu, s.lens, s.table, q, 0.125)
    n = int(s.cu[-1])
    assert np.all(np.abs(got - want)[:n] <= (2.0 ** -8 * np.abs(want) + bound)[:n])
    assert np.all(got[2 * new:n] == 0) and np.all(got[n:] == 9)
    assert np.all(got[new:2 * new - s.lens[1]] == 0) if s.lens[1] < new else True


@pytest.mark.parametrize("new", [1, 9, 100])
def test_attend_does_not_see_what_is_masked(tw, new):
    """Bytes behind the length, blocks that no row of a sequence sees and table entries behind it change
    nothing, whatever they hold; with a window neither do NaN scales in front of it."""
    import torch
    for window in (0, 70):
        s = Case(tw, 67, 128, 1, [new], [333])
        s.table = np.concatenate([s.table, np.full((1, 3), 10 ** 9, np.int32)], 1)
        q = dev(queries(s, 4), torch.bfloat16)
        c, b = s.device()
        first = host(tw.i8_kv_attend(c, b, q, window=window))
        total = 333 + new
        for side in (0, 1):
            tail = kv.place(side, 128)[(total - 1) % 64 + 1:].ravel()
            s.codes[s.table[0, (total - 1) // 64], :, side][:, tail] = -127
        unused = np.setdiff1d(np.arange(len(s.codes)), s.table[0])
        s.scales[unused] = np.nan
        if window:
            s.scales[s.table[0, :(333 - window + 1) // 64]] = np.nan
        c, b = s.device()
        assert np.array_equal(first, host(tw.i8_kv_attend(c, b, q, window=window)))
        assert np.isfinite(first).all()


@pytest.mark.parametrize("new", [1, 3, 130])
def test_attend_shows_what_is_not_finite(tw, new):
    """A NaN or infinite scale makes NaN exactly the rows that see the block; a query that is not
    finite makes NaN its own head only."""
    import torch
    for side, bad in ((0, np.nan), (1, np.nan), (0, np.inf), (1, np.inf)):
        s = Case(tw, 71, 64, 1, [new, new], [60, 200])
        s.codes[s.table[0, 0], :, side, :] = 0
        s.scales[s.table[0, 0], 0, side] = bad
        got = host(tw.i8_kv_attend(*s.device(), dev(queries(s, 2), torch.bfloat16)))
        assert np.isnan(got[:new]).all() and np.isfinite(got[new:]).all()
    s = Case(tw, 73, 64, 1, [new], [300])
    q = queries(s, 4)
    q[new // 2, 1, 5] = np.nan
    q[new // 2, 3, 6] = -np.inf
    got = host(tw.i8_kv_attend(*s.device(), dev(q, torch.bfloat16)))
    bad = np.isnan(got).all(-1)
    assert np.isnan(got).any(-1).sum() == bad.sum() == 2 and bad[new // 2, 1] and bad[new // 2, 3]


@pytest.mark.parametrize("new", [1, 5, 66])
def test_attend_missing_blocks(tw, new):
    s = Case(tw, 79, 64, 2, [new], [400])
    s.table[0, 1], s.table[0, 3] = -1, 10 ** 6
    check_attend(tw, s, queries(s, 4))
    # a table narrower than the length: what it does not hold is not seen
    s.table = s.table[:, :3].copy()
    check_attend(tw, s, queries(s, 4))


def test_attend_strided_rows_and_tables(tw):
    import torch
    s = Case(tw, 83, 128, 2, [3, 40], [100, 7])
    wide = dev(kv.bf16(s.rng.normal(size=(s.tokens, 12, 128))), torch.bfloat16)
    c, b = s.device()
    big = torch.full((2, s.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    big[:, :s.table.shape[1]] = b.table
    strided = tw.I8KvBatch(b.cu, b.lens, big[:, :s.table.shape[1]])
    a = tw.i8_kv_attend(c, strided, wide[:, 2:10])
    assert torch.equal(a, tw.i8_kv_attend(c, b, wide[:, 2:10].contiguous()))


@pytest.mark.parametrize("new, prev", [([1], [5000]), ([1] * 9, [300] * 9), ([12], [3000]), ([300], [2000])])
def test_attend_repeats_its_bytes_on_any_stream(tw, new, prev):
    import torch
    s = Case(tw, 89, 128, 2, new, prev)
    c, b = s.device()
    q = dev(queries(s, 8), torch.bfloat16)
    first = tw.i8_kv_attend(c, b, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        again = tw.i8_kv_attend(c, b, q, stream=side)
        both = tw.i8_kv_attend(c, b, q)
        torch.cuda.synchronize()
        assert torch.equal(first, again) and torch.equal(first, both)


def test_binding_refuses(tw):
    import torch
    c = tw.I8KvCache(2, 2, 64)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    b = tw.I8KvBatch(i32(0, 1), i32(1), i32(0).view(1, 1))
    f = tw.QkTransform(64)
    x = torch.zeros(1, 2, 64, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: tw.I8KvCache(2, 2, 96),
        lambda: tw.I8KvCache(codes=c.codes, scales=c.scales[:1]),
        lambda: tw.I8KvBatch(i32(0, 1).long(), i32(1), i32(0).view(1, 1)),
        lambda: tw.I8KvBatch(i32(0, 1), i32(1, 1), i32(0).view(1, 1)),
        lambda: tw.I8KvBatch(i32(0, 1), i32(1), i32(0)),
        lambda: tw.QkTransform(64, q_gain=torch.zeros(63, device="cuda")),
        lambda: tw.QkTransform(64, inv_freq=torch.zeros(32, device="cuda")),
        lambda: tw.qk_norm_rope(f, x.cpu(), None),
        lambda: tw.qk_norm_rope(f, x.double(), None),
        lambda: tw.qk_norm_rope(f, x, x.bfloat16()),
        lambda: tw.qk_norm_rope(tw.QkTransform(64, inv_freq=torch.zeros(32, dtype=torch.float64, device="cuda")),
                                x, None),
        lambda: tw.qk_norm_rope(f, x.transpose(0, 1), None, q_out=x),
        lambda: tw.qk_norm_rope(f, torch.zeros(2, 64, 2, device="cuda").transpose(1, 2), None),
        lambda: tw.i8_kv_append(c, b, tw.QkTransform(128), x, x),
        lambda: tw.i8_kv_append(c, b, f, x, x[:, :1]),
        lambda: tw.i8_kv_append(c, b, f, x, x.bfloat16()),
        lambda: tw.i8_kv_append(c, b, f, x, x, q=torch.zeros(1, 3, 64, device="cuda")),
        lambda: tw.i8_kv_append(c, b, f, x, x, q_out=q),
        lambda: tw.i8_kv_read(c, b, 1, dtype=torch.float16),
        lambda: tw.i8_kv_read(c, b, -1),
        lambda: tw.i8_kv_attend(c, b, q.float()),
        lambda: tw.i8_kv_attend(c, b, q[:, :3].contiguous()),
        lambda: tw.i8_kv_attend(c, b, q, out=q[:, :2]),
        lambda: tw.i8_kv_attend(c, b, q, window=-1),
        lambda: tw.i8_kv_attend(c, b, q, scale=float("nan")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(RuntimeError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_empty_calls(tw):
    import torch
    c = tw.I8KvCache(2, 2, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    b = tw.I8KvBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), none, none.view(0, 0))
    x = torch.zeros(0, 2, 64, device="cuda")
    q = tw.i8_kv_append(c, b, tw.QkTransform(64), x, x, q=x)
    assert tw.i8_kv_attend(c, b, q).shape == (0, 2, 64) and tw.i8_kv_read(c, b, 0)[0].shape == (0, 2, 64)
    assert tw.qk_norm_rope(tw.QkTransform(64), x, x)[1].shape == (0, 2, 64)


# ---- the step they make ----
def step_parts(tw, rng, hq, heads, d, hidden):
    n = (hq + 2 * heads) * d
    wqkv = tw.tern_pack(dev(synth.gen_ternary(rng, n, hidden)), dev(synth.gen_scales(rng, n, hidden // 128).view(np.int16)))
    wo = tw.tern_pack(dev(synth.gen_ternary(rng, hidden, hq * d)),
                      dev(synth.gen_scales(rng, hidden, hq * d // 128).view(np.int16)))
    qg, kg = rng.uniform(0.5, 1.5, (2, d)).astype(np.float32)
    f = tw.QkTransform(d, dev(qg), dev(kg), 1e-6, dev(F(d)))
    return n, wqkv, wo, qg, kg, f


def test_decode_steps_with_the_linears(tw):
    """q|k|v linear, append, attention, o linear over a prompt and then single tokens and a draft of
    four: every step's attention against the oracle run on the step's own linear outputs, and the
    cache's keys against their exact values."""
    import torch
    rng = np.random.default_rng(97)
    hq, heads, d, hidden = 8, 2, 128, 1024
    n, wqkv, wo, qg, kg, f = step_parts(tw, rng, hq, heads, d, hidden)
    cache = tw.I8KvCache(8, heads, d)
    table = dev(np.array([[5, 0, 7, 2]], np.int32))
    mirror = kv.Cache(np.zeros(cache.codes.shape, np.int8), np.zeros(cache.scales.shape, np.float32))
    length = 0
    for m in (61, 1, 1, 4, 1, 1):
        x = dev(synth.gen_x_bf16(rng, m, hidden).view(np.int16))
        if m > 16:
            y = tw.tern_gemm_prefill(wqkv, n, hidden, *tw.tern_quantize_i8(x))
        else:
            y = tw.tern_gemv(wqkv, n, hidden, x)
        rows = y.view(m, hq + 2 * heads, d)
        length += m
        cu, lens = np.array([0, m], np.int32), np.array([length], np.int32)
        batch = tw.I8KvBatch(dev(cu), dev(lens), table)
        q = tw.i8_kv_append(cache, batch, f, rows[:, hq:hq + heads], rows[:, hq + heads:], q=rows[:, :hq])
        out = tw.i8_kv_attend(cache, batch, q)
        z = tw.tern_gemv(wo, hidden, hq * d, out.view(m, -1)) if m <= 16 else None
        r = host(rows).astype(np.float64)
        pos = np.arange(length - m, length)
        key = kv.transform(r[:, hq:hq + heads], kg, 1e-6, F(d), False, pos)
        mirror.append(cu, lens, host(table), key, r[:, hq + heads:])
        # the library's cache and the exact one differ where a value sits on the border of two codes
        ks, vs = host(cache.scales), mirror.scales
        assert np.allclose(ks, vs, rtol=2.0 ** -18)
        assert np.abs(host(cache.codes).astype(int) - mirror.codes).max() <= 1
        own = kv.Cache(host(cache.codes), ks)
        want, bound = kv.attend(own, cu, lens, host(table), host(q), d ** -0.5)
        assert np.all(np.abs(host(out) - want) <= 2.0 ** -8 * np.abs(want) + bound)
        if z is not None:
            t = kv.bf16(host(out)).reshape(m, -1).view(np.uint32) >> 16
            y64, _ = oracle.gemv_bf16(host(wo), hidden, hq * d, t.astype(np.uint16))
            assert oracle.rel_l2(host(z), y64) <= 1e-5


def test_captured_step_follows_lengths(tw):
    """A captured step replayed while lens grows in place: every replay equals the eager calls on a
    second cache, with eager work and synchronisation in between."""
    import torch
    rng = np.random.default_rng(101)
    hq, heads, d, seqs = 8, 2, 128, 3
    f = tw.QkTransform(d, dev(rng.uniform(0.5, 1.5, d).astype(np.float32)), None, 1e-6, dev(F(d)))
    start = np.array([62, 900, 0], np.int32)
    table, blocks = pages(rng, start + 10, width=20)
    codes, scales = filled(rng, blocks, heads, d)
    made = [tw.I8KvCache(codes=dev(codes), scales=dev(scales)) for _ in range(2)]
    lens = [dev(start), dev(start)]
    cu = dev(np.arange(seqs + 1, dtype=np.int32))
    batches = [tw.I8KvBatch(cu, n, dev(table)) for n in lens]
    rows = torch.zeros(seqs, hq + 2 * heads, d, device="cuda")
    q = torch.empty(seqs, hq, d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = tw.i8_kv_attend_workspace(made[0], batches[0], seqs, hq)

    def step(i, q, out, ws):
        lens[i] += 1
        tw.i8_kv_append(made[i], batches[i], f, rows[:, hq:hq + heads], rows[:, hq + heads:], q=rows[:, :hq],
                        q_out=q)
        tw.i8_kv_attend(made[i], batches[i], q, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0, q, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0, q, out, ws)
    lens[0].copy_(dev(start))                       # the warm-up step and the capture: start over
    made[0].codes.copy_(dev(codes))
    made[0].scales.copy_(dev(scales))
    for i in range(6):
        rows.copy_(dev(rng.normal(size=tuple(rows.shape)).astype(np.float32) * 1.5 ** i))
        graph.replay()
        qe, oe = torch.empty_like(q), torch.empty_like(out)
        step(1, qe, oe, None)
        torch.cuda.synchronize()
        assert torch.equal(q, qe) and torch.equal(out, oe)
        assert torch.equal(made[0].codes, made[1].codes) and torch.equal(made[0].scales, made[1].scales)


def test_far_blocks_of_a_large_cache(tw):
    """Blocks whose bytes lie past 2^32: 64-bit addresses throughout."""
    import torch
    d, heads = 128, 8
    blocks = 2 ** 32 // (heads * 2 * 64 * d) + 40
    codes = torch.zeros((blocks, heads, 2, 64 * d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((blocks, heads, 2), device="cuda")
    c = tw.I8KvCache(codes=codes, scales=scales)
    table = torch.tensor([[blocks - 1, 3, blocks - 7, blocks // 2]], dtype=torch.int32, device="cuda")
    low = tw.I8KvCache(4, heads, d)
    order = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    rng = np.random.default_rng(5)
    k, v = dev(rng.normal(size=(2, 250, heads, d)).astype(np.float32))
    q = dev(rng.normal(size=(250, 16, d)), torch.bfloat16)
    cu, lens = dev(np.array([0, 250], np.int32)), dev(np.array([250], np.int32))
    got = []
    for cache, t in ((c, table), (low, order)):
        b = tw.I8KvBatch(cu, lens, t)
        tw.i8_kv_append(cache, b, tw.QkTransform(d), k, v)
        one = tw.I8KvBatch(dev(np.array([0, 1], np.int32)), lens, t)
        got.append((tw.i8_kv_attend(cache, b, q), tw.i8_kv_attend(cache, one, q[:1]), *tw.i8_kv_read(cache, b, 250)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
