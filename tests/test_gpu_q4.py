"""4-bit weights with group scales on the GPU against the 64-bit oracle
(oracle/q4.py): the blob's bytes, and products within the oracle's bound on
every output."""
import numpy as np
import pytest

import ternary_weight_decode_amd as tw
from oracle import kv, q4

from test_gpu_kv import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    assert torch.cuda.is_available()
    tw.lib()


def host(t):
    import torch
    torch.cuda.synchronize()
    return t.cpu().numpy()


def weights(rng, n, k, group):
    t = np.clip(np.rint(rng.normal(size=(n, k)) * 3.2), -8, 7).astype(np.int8)
    return t, rng.uniform(0.002, 0.05, (n, k // group)).astype(np.float16)


def bf16_bits(x):
    return (kv.bf16(x).view(np.uint32) >> 16).astype(np.uint16).view(np.int16)


@pytest.mark.parametrize("n, k, group", [(16, 128, 128), (1, 128, 32), (37, 640, 64), (33, 1408, 32), (100, 1024, 128)])
def test_pack_bytes(n, k, group):
    rng = np.random.default_rng([n, k])
    t, s = weights(rng, n, k, group)
    t = rng.integers(-128, 128, (n, k)).astype(np.int8) if n == 37 else t       # clamped
    assert np.array_equal(host(tw.q4_pack(dev(t), dev(s))), q4.pack(t, s))


# one row tile and many, K of one block to more than any wave holds, k-tiles
# that end early, every count of rows
SHAPES = [(1, 128, 32, 1), (16, 256, 64, 2), (17, 384, 128, 16), (40, 512, 32, 4), (300, 640, 64, 1), (64, 1024, 32, 3),
          (100, 1152, 32, 13), (1000, 2048, 128, 1), (513, 4096, 64, 5), (2050, 4096, 128, 8), (33, 12288, 64, 7),
          (48, 20480, 32, 16), (31, 33408, 128, 2), (4096, 1024, 32, 1), (9000, 512, 128, 6), (24576, 256, 64, 1)]


@pytest.mark.parametrize("n, k, group, m", SHAPES)
def test_products(n, k, group, m):
    import torch
    rng = np.random.default_rng([n, k, m])
    t, s = weights(rng, n, k, group)
    packed = tw.q4_pack(dev(t), dev(s))
    # channels of unequal size, rows with a mean
    x = kv.bf16(rng.normal(size=(m, k)) * np.exp(rng.normal(size=(1, k))) + rng.normal(size=(m, 1)))
    got = host(tw.q4_gemv(packed, n, k, group, dev(x, torch.bfloat16)))
    want, bound = q4.gemv(t, s, x)
    assert got.shape == (m, n) and np.all(np.abs(got - want) <= bound)
    q, sx = rng.integers(-127, 128, (m, k)).astype(np.int8), rng.uniform(0.001, 0.1, m).astype(np.float32)
    got = host(tw.q4_gemv_i8(packed, n, k, group, dev(q), dev(sx)))
    want, bound = q4.gemv_i8(t, s, q, sx)
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("n, k, group, m", [(40, 1024, 32, 1), (40, 1024, 128, 3), (40, 640, 64, 11)])
def test_activations_of_every_size(n, k, group, m):
    """Rows of nothing but zeros, of the smallest and the largest values, and with one value 2^30 times the rest
    (its weights 0 in half of the outputs): each within its own bound."""
    import torch
    rng = np.random.default_rng([k, m])
    t, s = weights(rng, n, k, group)
    t[::2, 5] = 0
    packed = tw.q4_pack(dev(t), dev(s))
    for size in (0.0, 2.0 ** -126, 2.0 ** -133, 2.0 ** -110, 2.0 ** 60, 2.0 ** 112, None):
        x = rng.normal(size=(m, k)) * (1.0 if size is None else size)
        if size is None:
            x[:, 5] = 2.0 ** 30
        x = kv.bf16(x)
        got = host(tw.q4_gemv(packed, n, k, group, dev(bf16_bits(x))))
        want, bound = q4.gemv(t, s, x)
        # below fp32's normal numbers a result has a step of 2^-149, a product with a scale too
        assert np.all(np.abs(got - want) <= bound + (k // group + 20) * 2.0 ** -149), size


@pytest.mark.parametrize("m", [1, 4, 16])
def test_rows_that_are_not_finite(m):
    import torch
    rng = np.random.default_rng(m)
    n, k, group = 50, 1152, 32
    t, s = weights(rng, n, k, group)
    packed = tw.q4_pack(dev(t), dev(s))
    x = kv.bf16(rng.normal(size=(m, k)))
    clean = host(tw.q4_gemv(packed, n, k, group, dev(x, torch.bfloat16)))
    for bad in (np.inf, -np.inf, np.nan):
        y = x.copy()
        y[m // 2, 700] = bad
        got = host(tw.q4_gemv(packed, n, k, group, dev(y, torch.bfloat16)))
        assert not np.isfinite(got[m // 2]).any()
        rest = np.arange(m) != m // 2
        assert np.array_equal(got[rest], clean[rest])


@pytest.mark.parametrize("m", [1, 2, 9])
def test_largest_sums(m):
    """Every product at its largest, of one sign: nothing overflows on the way."""
    import torch
    n, k, group = 20, 4096, 128
    t = np.full((n, k), -8, np.int8)
    s = np.full((n, k // group), 60000.0, np.float16)
    packed = tw.q4_pack(dev(t), dev(s))
    q, sx = np.full((m, k), -127, np.int8), np.full(m, 3.0, np.float32)
    assert np.allclose(host(tw.q4_gemv_i8(packed, n, k, group, dev(q), dev(sx))), q4.gemv_i8(t, s, q, sx)[0], rtol=1e-5)
    x = kv.bf16(np.full((m, k), 2.0 ** 90))
    assert np.allclose(host(tw.q4_gemv(packed, n, k, group, dev(x, torch.bfloat16))), q4.gemv(t, s, x)[0], rtol=1e-5)


def test_equal_calls_equal_bytes_and_nothing_else_written():
    import torch
    rng = np.random.default_rng(7)
    for n, k, group, m in [(35, 1408, 32, 3), (500, 4096, 128, 1), (70, 12288, 64, 16)]:
        t, s = weights(rng, n, k, group)
        packed, x = tw.q4_pack(dev(t), dev(s)), dev(rng.normal(size=(m, k)).astype(np.float32), torch.bfloat16)
        room = torch.full((m * n + 64,), 7.0, device="cuda")
        y = room[32:32 + m * n].view(m, n)
        one = tw.q4_gemv(packed, n, k, group, x)
        tw.q4_gemv(packed, n, k, group, x, y=y)
        assert torch.equal(one, y) and bool((room[:32] == 7).all()) and bool((room[32 + m * n:] == 7).all())


def test_captured_and_on_another_stream():
    """Two products in a graph on a stream of their own, replayed with other inputs between eager work."""
    import torch
    rng = np.random.default_rng(11)
    n, k, group = 700, 2048, 64
    t, s = weights(rng, n, k, group)
    packed = tw.q4_pack(dev(t), dev(s))
    xs = [dev(rng.normal(size=(2, k)).astype(np.float32), torch.bfloat16) for _ in range(3)]
    qs = [tw.tern_quantize_i8(x) for x in xs]
    want = [(tw.q4_gemv(packed, n, k, group, x), tw.q4_gemv_i8(packed, n, k, group, *q)) for x, q in zip(xs, qs)]
    x, q, sx = xs[0].clone(), qs[0][0].clone(), qs[0][1].clone()
    y, yi = torch.empty(2, n, device="cuda"), torch.empty(2, n, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(tw.q4_gemv(packed, n, k, group, x, stream=side), want[0][0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tw.q4_gemv(packed, n, k, group, x, y=y)
        tw.q4_gemv_i8(packed, n, k, group, q, sx, y=yi)
    for i in (0, 2, 1, 1, 0):
        x.copy_(xs[i]), q.copy_(qs[i][0]), sx.copy_(qs[i][1])
        y.zero_(), yi.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(yi, want[i][1])


@pytest.mark.parametrize("m", [1, 5, 16])
def test_row_scales_of_every_size(m):
    """Scales of activations down to fp32's smallest number and up to where results leave it."""
    rng = np.random.default_rng(m)
    n, k, group = 50, 1152, 32
    t, s = weights(rng, n, k, group)
    packed = tw.q4_pack(dev(t), dev(s))
    q = rng.integers(-127, 128, (m, k)).astype(np.int8)
    for size in (2.0 ** -149, 13 * 2.0 ** -149, 2.0 ** -130 * 1.37, 2.0 ** -126, 1e-30, 1.0, 2.0 ** 100):
        sx = np.full(m, size, np.float32)
        got = host(tw.q4_gemv_i8(packed, n, k, group, dev(q), dev(sx)))
        want, bound = q4.gemv_i8(t, s, q, sx)
        # a result below fp32's normal numbers has a step of 2^-149
        assert np.all(np.abs(got - want) <= bound + 2.0 ** -149), size
