"""The 4-bit and tree calls refuse bad arguments on the host, before any HIP
call (no GPU): every call here passes addresses that are never dereferenced."""
import ctypes
import itertools

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


def attend(c=None, b=None, T=1, q=P, hq=4, qs=512, scale=0.1, mask=P, words=1, max_len=256, out=P, ws=P):
    return tw.lib().i8_kv_attend_tree(ctypes.byref(c or cache()), ctypes.byref(b or batch()), T, q, hq, qs, scale,
                                      mask, words, max_len, out, ws, None)


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
    (dict(qs=504), E_SHAPE), (dict(max_len=0), E_SHAPE), (dict(c=cache(d=32)), E_SHAPE),
    (dict(mask=None), E_NULL), (dict(q=None), E_NULL), (dict(out=None), E_NULL), (dict(mask=ODD), E_ALIGN),
    (dict(q=ODD), E_ALIGN), (dict(out=ODD), E_ALIGN), (dict(T=0, mask=None), E_OK),
])
def test_attend_refuses(kw, rc):
    assert attend(**kw) == rc


@pytest.mark.parametrize("hq, heads, d", [(32, 8, 128), (16, 8, 128), (1, 1, 64), (20, 1, 128)])
def test_attend_plan(hq, heads, d):
    """Every unit has a workgroup, cut or not, and the workspace is what the cut takes."""
    for rows, nseq, width in itertools.product((1, 7, 64, 500, 5000), (1, 2, 70, 2000), (0, 1, 30, 700, 20000)):
        p = tw.i8_kv_attend_tree_config(rows, hq, heads, d, nseq, width)
        units = (rows * (hq // heads) // p["cols"] + nseq) * heads
        assert p["cols"] in (16, 128), (rows, nseq, width, p)
        assert p["groups"] in ((0, 768) if p["cols"] == 16 else (0, 256, 512)), (rows, nseq, width, p)
        assert p["grid"] == units + p["groups"] and not (p["cols"] == 128 and p["groups"] and units > 1024)
        need = tw.i8_kv_attend_tree_workspace_bytes(rows, hq, heads, d, nseq, max(1, 64 * width))
        used = p["grid"] * p["cols"] * (4 * d + 8) + (nseq + 5) // 4 * 16 if p["groups"] else 0
        # lengths that would pass 32 bits in the line stay whole, whatever the workspace
        assert used == need or units * width > 2 ** 30, (rows, nseq, width, p, used, need)
    wide = (2 ** 31 - 1) // 64
    assert tw.i8_kv_attend_tree_config(64, hq, heads, d, 1, 1000)["groups"] > 0
    assert tw.i8_kv_attend_tree_config(64, 32, 8, d, 64, wide, 64000)["groups"] == 0
    assert tw.i8_kv_attend_tree_config(0, hq, heads, d, 1, 5) == {} == tw.i8_kv_attend_tree_config(5, hq, heads, d, 0, 5)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(hq=3), dict(heads=0), dict(d=96), dict(nseq=-1), dict(width=-1),
                                 dict(width=2 ** 26), dict(max_len=0), dict(max_len=2 ** 31)])
def test_attend_plan_refuses(bad):
    with pytest.raises(RuntimeError):
        tw.i8_kv_attend_tree_config(**{**dict(tokens=8, hq=4, heads=2, d=64, nseq=2, width=9), **bad})


@pytest.mark.parametrize("call", [mask, accept])
def test_a_batch_without_lengths_is_refused(call):
    """The batch's three arrays, whichever of them a call reads."""
    assert call(b=batch(lens=None)) == E_NULL
    assert call(b=batch(lens=P + 2)) == E_ALIGN
    assert call(b=batch(cu=P + 2)) == E_ALIGN


@pytest.mark.parametrize("hq, heads, d", [(32, 8, 128), (16, 8, 64), (1, 1, 64), (20, 1, 128), (800, 800, 64), (64, 2, 64)])
def test_one_workspace_serves_smaller_calls(hq, heads, d):
    """Sizes of a call and of those below it, in which chunks come and go: the limit holds all of them, and grows
    with the sizes."""
    need, limit = tw.i8_kv_attend_tree_workspace_bytes, tw.i8_kv_attend_tree_workspace_limit
    lengths = (1, 64, 500, 2000, 8000, 16000, 60000, 10 ** 6, 2 ** 31 - 1)
    sizes = sorted({int(1.3 ** i) for i in range(45)} | {24 * i for i in range(0, 200, 7)} | {0, 2000, 5000})
    most = {}                                   # of any call of these rows, by sequences
    for rows in sizes:
        if rows * hq > 2 ** 25:
            break
        for nseq in (0, 1, 2, 3, 5, 8, 17, 32, 47, 64, 90, 100, 128, 140, 378, 756, 1024, 3000):
            largest = max(need(rows, hq, heads, d, nseq, n) for n in lengths)
            for other, seen in most.items():
                if other <= nseq:
                    largest = max(largest, seen)
            most[nseq] = max(most.get(nseq, 0), largest)
            assert limit(rows, hq, heads, d, nseq) >= most[nseq], (rows, nseq)
            if rows and nseq:
                assert limit(rows, hq, heads, d, nseq) >= limit(max(1, rows - 1), hq, heads, d, max(1, nseq - 1))
    assert limit(0, hq, heads, d, 5) == 0 == limit(5, hq, heads, d, 0)


def test_the_limit_refuses():
    for kw in (dict(tokens=-1), dict(hq=3), dict(heads=0), dict(d=96), dict(nseq=-1), dict(tokens=2 ** 24)):
        assert tw.i8_kv_attend_tree_workspace_limit(**{**dict(tokens=8, hq=4, heads=2, d=64, nseq=2), **kw}) == -1
