"""The 4-bit and tree calls refuse bad arguments on the host, before any HIP
call (no GPU): every call here passes addresses that are never dereferenced."""
import ctypes

import pytest

import ternary_weight_decode_amd as tw

from test_kv_abi import batch, cache

E_OK, E_NULL, E_SHAPE, E_ALIGN = 0, 1, 2, 3
P, ODD = 0x10000, 0x10004


def pack(t=P, scale=P, n=16, k=128, group=64, packed=P):
    return tw.lib().q4_pack(t, scale, n, k, group, packed, None)


def gemv(packed=P, n=16, k=128, group=64, x=P, m=1, y=P):
    return tw.lib().q4_gemv(packed, n, k, group, x, m, y, None)


def gemv_i8(packed=P, n=16, k=128, group=64, q=P, s=P, m=1, y=P):
    return tw.lib().q4_gemv_i8(packed, n, k, group, q, s, m, y, None)


def mask(b=None, T=1, parent=P, words=1, mask=P, pos=P, no_b=False):
    return tw.lib().draft_tree_mask(None if no_b else ctypes.byref(b or batch()), T, parent, words, mask, pos, None)


def accept(b=None, T=1, parent=P, token=P, target=P, width=4, path=P, count=P, following=P, no_b=False):
    return tw.lib().draft_tree_accept(None if no_b else ctypes.byref(b or batch()), T, parent, token, target, width,
                                      path, count, following, None)


def keep(c=None, b=None, T=1, path=P, width=4, lens=P, nulls=()):
    ref = lambda name, x: None if name in nulls else ctypes.byref(x)
    return tw.lib().i8_kv_keep(ref("c", c or cache()), ref("b", b or batch()), T, path, width, lens, None)


def attend(c=None, b=None, T=1, q=P, hq=4, qs=512, scale=0.1, mask=P, words=1, max_len=256, max_rows=0, out=P, ws=P):
    return tw.lib().i8_kv_attend_tree(ctypes.byref(c or cache()), ctypes.byref(b or batch()), T, q, hq, qs, scale,
                                      mask, words, max_len, max_rows, out, ws, None)


BAD = [(dict(n=-1), E_SHAPE), (dict(k=64), E_SHAPE), (dict(k=-128), E_SHAPE), (dict(group=48), E_SHAPE),
       (dict(group=0), E_SHAPE), (dict(group=256), E_SHAPE), (dict(packed=None), E_NULL), (dict(packed=ODD), E_ALIGN),
       (dict(n=0, packed=None), E_OK)]
PRODUCT = BAD + [(dict(m=-1), E_SHAPE), (dict(m=17), E_SHAPE), (dict(n=1 << 29), E_SHAPE),
                 (dict(k=1 << 25), E_SHAPE), (dict(y=None), E_NULL),
                 (dict(y=P + 2), E_ALIGN), (dict(m=0, y=None), E_OK)]


@pytest.mark.parametrize("kw, rc", BAD + [(dict(t=None), E_NULL), (dict(scale=None), E_NULL), (dict(t=ODD), E_ALIGN),
                                          (dict(scale=P + 1), E_ALIGN), (dict(k=0, t=None), E_OK)])
def test_pack_refuses(kw, rc):
    assert pack(**kw) == rc


@pytest.mark.parametrize("kw, rc", PRODUCT + [(dict(x=None), E_NULL), (dict(x=ODD), E_ALIGN)])
def test_gemv_refuses(kw, rc):
    assert gemv(**kw) == rc


@pytest.mark.parametrize("kw, rc", PRODUCT + [(dict(q=None), E_NULL), (dict(q=ODD), E_ALIGN), (dict(s=None), E_NULL),
                                              (dict(s=P + 2), E_ALIGN)])
def test_gemv_i8_refuses(kw, rc):
    assert gemv_i8(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(no_b=True), E_NULL), (dict(T=-1), E_SHAPE), (dict(T=1 << 25), E_SHAPE), (dict(words=0), E_SHAPE),
    (dict(words=9), E_SHAPE), (dict(b=batch(nseq=-1)), E_SHAPE), (dict(b=batch(cu=None)), E_NULL),
    (dict(b=batch(lens=None)), E_NULL), (dict(parent=None), E_NULL), (dict(mask=None), E_NULL),
    (dict(mask=ODD), E_ALIGN), (dict(pos=P + 2), E_ALIGN), (dict(parent=P + 2), E_ALIGN),
    (dict(T=0, parent=None, mask=None), E_OK), (dict(b=batch(nseq=0), mask=None), E_OK),
])
def test_mask_refuses(kw, rc):
    assert mask(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(no_b=True), E_NULL), (dict(T=-1), E_SHAPE), (dict(width=0), E_SHAPE), (dict(width=1 << 17), E_SHAPE),
    (dict(b=batch(cu=None)), E_NULL), (dict(parent=None), E_NULL), (dict(token=None), E_NULL),
    (dict(target=None), E_NULL), (dict(path=None), E_NULL), (dict(path=P + 2), E_ALIGN), (dict(token=P + 1), E_ALIGN),
    (dict(count=P + 2), E_ALIGN), (dict(following=P + 2), E_ALIGN), (dict(b=batch(nseq=0), path=None), E_OK),
])
def test_accept_refuses(kw, rc):
    assert accept(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(nulls=("c",)), E_NULL), (dict(nulls=("b",)), E_NULL), (dict(T=-1), E_SHAPE), (dict(width=0), E_SHAPE),
    (dict(c=cache(d=96)), E_SHAPE), (dict(c=cache(heads=0)), E_SHAPE), (dict(b=batch(stride=3)), E_SHAPE),
    (dict(path=None), E_NULL), (dict(c=cache(codes=None)), E_NULL), (dict(b=batch(table=None)), E_NULL),
    (dict(path=P + 2), E_ALIGN), (dict(lens=P + 2), E_ALIGN), (dict(c=cache(codes=ODD)), E_ALIGN),
    (dict(b=batch(nseq=0), path=None), E_OK),
])
def test_keep_refuses(kw, rc):
    assert keep(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(words=0), E_SHAPE), (dict(words=9), E_SHAPE), (dict(hq=3), E_SHAPE), (dict(scale=float("nan")), E_SHAPE),
    (dict(qs=504), E_SHAPE), (dict(max_len=0), E_SHAPE), (dict(max_rows=-1), E_SHAPE), (dict(c=cache(d=32)), E_SHAPE),
    (dict(mask=None), E_NULL), (dict(q=None), E_NULL), (dict(out=None), E_NULL), (dict(mask=ODD), E_ALIGN),
    (dict(q=ODD), E_ALIGN), (dict(out=ODD), E_ALIGN), (dict(T=0, mask=None), E_OK),
])
def test_attend_refuses(kw, rc):
    assert attend(**kw) == rc
