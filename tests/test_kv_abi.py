"""The cache calls refuse bad arguments on the host, before any HIP call (no
GPU): every call here passes addresses that are never dereferenced."""
import ctypes

import pytest

import ternary_weight_decode_amd as tw

E_OK, E_NULL, E_SHAPE, E_ALIGN = 0, 1, 2, 3
P, ODD = 0x10000, 0x10004
BF16, F32 = 1, 0


def cache(codes=P, scales=P, blocks=4, heads=2, d=128):
    return tw._KvCache(codes, scales, blocks, heads, d)


def batch(cu=P, lens=P, table=P, nseq=1, width=4, stride=4):
    return tw._KvBatch(cu, lens, table, nseq, width, stride)


def transform(q_gain=P, k_gain=P, inv_freq=P):
    return tw._QkTransform(q_gain, k_gain, inv_freq, 1e-6, 0)


def norm(f=None, T=1, d=128, q=P, hq=4, qs=512, k=P, hk=2, ks=256, it=F32, pos=P, qo=P, ko=P, ot=BF16, no_f=False):
    f = None if no_f else ctypes.byref(f or transform())
    return tw.lib().qk_norm_rope(f, T, d, q, hq, qs, k, hk, ks, it, pos, qo, ko, ot, None)


def append(c=None, b=None, f=None, T=1, q=P, hq=4, qs=512, k=P, ks=256, v=P, vs=256, it=F32, pos=P, qo=P,
           nulls=()):
    ref = lambda name, x: None if name in nulls else ctypes.byref(x)
    return tw.lib().i8_kv_append(ref("c", c or cache()), ref("b", b or batch()), ref("f", f or transform()), T, q, hq,
                                 qs, k, ks, v, vs, it, pos, qo, None)


def read(c=None, b=None, T=1, ko=P, vo=P, ot=BF16):
    return tw.lib().i8_kv_read(ctypes.byref(c or cache()), ctypes.byref(b or batch()), T, ko, vo, ot, None)


def attend(c=None, b=None, T=1, q=P, hq=4, qs=512, scale=0.1, window=0, max_len=256, max_rows=0, out=P, ws=P):
    return tw.lib().i8_kv_attend(ctypes.byref(c or cache()), ctypes.byref(b or batch()), T, q, hq, qs, scale, window,
                                 max_len, max_rows, out, ws, None)


@pytest.mark.parametrize("kw, rc", [
    (dict(d=96), E_SHAPE), (dict(d=0), E_SHAPE), (dict(T=-1), E_SHAPE), (dict(hq=-1), E_SHAPE),
    (dict(T=1 << 25), E_SHAPE), (dict(hq=1025, qs=1 << 20), E_SHAPE), (dict(it=2), E_SHAPE), (dict(ot=-1), E_SHAPE),
    (dict(qs=508), E_SHAPE), (dict(ks=255), E_SHAPE), (dict(qs=513), E_SHAPE), (dict(it=BF16, qs=516), E_SHAPE),
    (dict(no_f=True), E_NULL), (dict(q=None), E_NULL), (dict(ko=None), E_NULL), (dict(pos=None), E_NULL),
    (dict(q=ODD), E_ALIGN), (dict(k=ODD), E_ALIGN), (dict(qo=ODD), E_ALIGN), (dict(pos=P + 1), E_ALIGN),
    (dict(f=transform(q_gain=ODD)), E_ALIGN), (dict(f=transform(inv_freq=P + 4)), E_ALIGN),
    (dict(T=0, q=None, k=None), E_OK), (dict(hq=0, hk=0), E_OK),
])
def test_norm_refuses(kw, rc):
    assert norm(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(c=cache(d=80)), E_SHAPE), (dict(c=cache(heads=0)), E_SHAPE), (dict(c=cache(blocks=-1)), E_SHAPE),
    (dict(b=batch(nseq=-1)), E_SHAPE), (dict(b=batch(width=-1)), E_SHAPE), (dict(b=batch(stride=3)), E_SHAPE),
    (dict(T=-1), E_SHAPE), (dict(T=(1 << 24) + 1), E_SHAPE), (dict(hq=3), E_SHAPE), (dict(hq=-2), E_SHAPE),
    (dict(ks=252), E_SHAPE), (dict(vs=257), E_SHAPE), (dict(qs=511), E_SHAPE), (dict(it=7), E_SHAPE),
    (dict(nulls="c"), E_NULL), (dict(nulls="b"), E_NULL), (dict(nulls="f"), E_NULL), (dict(k=None), E_NULL),
    (dict(v=None), E_NULL), (dict(q=None), E_NULL), (dict(qo=None), E_NULL), (dict(c=cache(codes=None)), E_NULL),
    (dict(c=cache(scales=None)), E_NULL), (dict(b=batch(cu=None)), E_NULL), (dict(b=batch(lens=None)), E_NULL),
    (dict(b=batch(table=None)), E_NULL), (dict(c=cache(codes=ODD)), E_ALIGN), (dict(k=ODD), E_ALIGN),
    (dict(v=ODD), E_ALIGN), (dict(q=ODD), E_ALIGN), (dict(qo=ODD), E_ALIGN), (dict(b=batch(cu=P + 2)), E_ALIGN),
    (dict(pos=P + 2), E_ALIGN), (dict(f=transform(k_gain=ODD)), E_ALIGN),
    (dict(T=0, k=None, v=None), E_OK), (dict(b=batch(nseq=0, lens=None)), E_OK),
])
def test_append_refuses(kw, rc):
    assert append(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(c=cache(d=32)), E_SHAPE), (dict(ot=3), E_SHAPE), (dict(T=-3), E_SHAPE), (dict(ko=None), E_NULL),
    (dict(vo=None), E_NULL), (dict(ko=ODD), E_ALIGN), (dict(vo=ODD), E_ALIGN), (dict(T=0, ko=None), E_OK),
])
def test_read_refuses(kw, rc):
    assert read(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(c=cache(d=256)), E_SHAPE), (dict(hq=5), E_SHAPE), (dict(hq=0), E_SHAPE), (dict(qs=504), E_SHAPE),
    (dict(qs=516), E_SHAPE), (dict(window=-1), E_SHAPE), (dict(max_len=0), E_SHAPE),
    (dict(max_rows=-1), E_SHAPE),
    (dict(scale=float("nan")), E_SHAPE), (dict(scale=float("inf")), E_SHAPE), (dict(T=-1), E_SHAPE),
    (dict(q=None), E_NULL), (dict(out=None), E_NULL), (dict(q=ODD), E_ALIGN), (dict(out=ODD), E_ALIGN),
    (dict(b=batch(lens=P + 1)), E_ALIGN), (dict(T=0, q=None), E_OK), (dict(b=batch(nseq=0)), E_OK),
])
def test_attend_refuses(kw, rc):
    assert attend(**kw) == rc


def test_workspace_sizes():
    ws = tw.i8_kv_attend_workspace_bytes        # max_rows 0: not known
    assert ws(1, 4, 3, 128, 1, 64) == -1 and ws(1, 4, 2, 96, 1, 64) == -1 and ws(-1, 4, 2, 128, 1, 64) == -1
    assert ws(1, 4, 2, 128, 1, 0) == -1 and ws(1, 0, 2, 128, 1, 64) == -1
    assert ws(0, 4, 2, 128, 1, 64) == 0 and ws(5, 4, 2, 128, 0, 64) == 0
    assert ws(1, 4, 2, 128, 1, 64, -1) == -1 and ws(1 << 24, 4, 2, 128, 1, 64) == -1
    assert ws(1, 32, 8, 128, 1, 40960) > 0 and ws(1, 32, 8, 128, 1, 512) == 0
    # a batch that may hold prompts beside single tokens works in two launches, told otherwise in one
    assert ws(2111, 32, 8, 128, 64, 8192) > ws(2111, 32, 8, 128, 64, 8192, 16)
    # the split is bounded, whatever the hint
    assert ws(4096, 32, 8, 128, 4096, 10 ** 6) < 1 << 30
