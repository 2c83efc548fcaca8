"""Batches whose cu descends: the sequences in front of the descent are served
as if they were alone, nothing behind it is read or written."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import kv

from test_gpu_kv import Case, dev, host, queries
from test_gpu_kv_tile import LONG, exact

pytestmark = pytest.mark.gpu


def broken(s, cu, lens, rows):
    """The case's sequences in a batch of this cu, their tables again for those behind."""
    n = len(s.lens)
    table = np.resize(s.table, (len(lens), s.table.shape[1]))
    table[:n] = s.table
    return tw.I8KvBatch(dev(np.array(cu, np.int32)), dev(np.array(lens, np.int32)), dev(table))


@pytest.mark.parametrize("new, prev, max_len, cols, groups", [
    ([20, 3], [100, 30], None, 16, False), ([20, 3], [3000, 40], None, 16, True),
    ([300, 200], [700, 30], LONG, 256, True), ([300, 3], [700, 3000], LONG, 256, True),
])
def test_attend_up_to_a_descent(new, prev, max_len, cols, groups):
    import torch
    s = Case(tw, 500 + prev[0], 64, 2, new, prev, spare_rows=30)
    q = queries(s, 8)
    n = int(s.cu[-1])
    cu = [0, new[0], n, n - 1, n, 2, n + 20, n + 30]
    lens = [*s.lens, 64, 64, 500, 500, 500]
    launches = tw.i8_kv_attend_config(s.tokens, 8, 2, 64, len(lens), s.table.shape[1], max_len=max_len)
    assert launches[0]["cols"] == cols and bool(launches[0]["groups"]) == groups
    out = torch.full((s.tokens, 8, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    c = s.device()[0]
    tw.i8_kv_attend(c, broken(s, cu, lens, s.tokens), dev(q, torch.bfloat16), max_len=max_len, out=out)
    got = host(out)
    want, bound = exact(s, q)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[:n])
    assert np.all(got[n:] == 9)


@pytest.mark.parametrize("max_rows", [0, 512])
def test_attend_the_same_rows_a_thousand_times(max_rows):
    """Taken one by one, the sequences' blocks would number far past 2^32."""
    import torch
    seqs = 2000
    s = Case(tw, 510, 64, 8, [512], [1000])
    q = queries(s, 32)
    wide = np.full((1, 32000), -1, np.int32)
    wide[:, :s.table.shape[1]] = s.table
    cu = [0, 512] * (seqs // 2) + [0]
    table = dev(np.broadcast_to(wide, (seqs, wide.shape[1])))
    b = tw.I8KvBatch(dev(np.array(cu, np.int32)), dev(np.array([int(s.lens[0])] + [32000 * 64 - 1] * (seqs - 1), np.int32)),
                     table)
    launches = tw.i8_kv_attend_config(s.tokens, 32, 8, 64, seqs, wide.shape[1], max_rows=max_rows)
    assert len(launches) == (2 if max_rows else 1) and launches[-1]["groups"]
    got = host(tw.i8_kv_attend(s.device()[0], b, dev(q, torch.bfloat16), max_rows=max_rows))
    s.table = wide
    want, bound = exact(s, q, rows=np.arange(0, 512, 37))
    rows = np.arange(0, 512, 37)
    assert np.all((np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + bound)[rows])


def test_append_and_read_up_to_a_descent():
    """Many blocks in front of the descent, and sequences behind it whose items would fall among them."""
    import torch
    new, prev = [1000, 70], [30, 100]
    s = Case(tw, 520, 64, 2, new, prev, spare_rows=5)
    cu = [0, 1000, 1070, 40, 900, 1075]
    lens = [*s.lens, 64, 900, 300]
    b = broken(s, cu, lens, s.tokens)
    k, v = s.rng.normal(size=(2, s.tokens, 2, 64)).astype(np.float32)
    c = s.device()[0]
    q_out = torch.full((s.tokens, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    tw.i8_kv_append(c, b, tw.QkTransform(64), dev(k), dev(v), q=dev(k), q_out=q_out)
    want = kv.Cache(s.codes, s.scales)
    want.append(s.cu, s.lens, s.table, k, v)
    assert np.array_equal(host(c.scales), want.scales) and np.array_equal(host(c.codes), want.codes)
    assert np.array_equal(host(q_out)[:1070], kv.bf16(k[:1070])) and np.all(host(q_out)[1070:] == 5)
    outs = torch.full((2, s.tokens, 2, 64), 3.0, device="cuda")
    tw.i8_kv_read(c, b, s.tokens, k_out=outs[0], v_out=outs[1])
    for got, w in zip(host(outs), want.read(s.cu, s.lens, s.table, s.tokens)):
        assert np.array_equal(got[:1070], w[:1070].astype(np.float32)) and np.all(got[1070:] == 3)
