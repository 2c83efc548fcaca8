"""Host side of the 4-bit and tree calls' binding, with the library and the
allocator stood in for (no GPU): names, memory, checks of tensors."""
import inspect
import types

import pytest
import torch

import ternary_weight_decode_amd as tw
from ternary_weight_decode_amd import draft_tree, q4

HELD = (q4, draft_tree)


def test_the_package_has_the_submodules_names():
    for module in HELD:
        for name, f in vars(module).items():
            if inspect.isfunction(f) and not name.startswith("_"):
                assert getattr(tw, name) is f and name in dir(tw), name
    assert tw.TREE_ROWS == 512
    with pytest.raises(AttributeError):
        tw.no_such_call


class Tensor(torch.Tensor):
    """A host tensor that passes for one on device 0."""
    is_cuda = True

    def get_device(self):
        return 0


def fake(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Tensor)


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library, and the streams that memory was taken from."""
    seen = {"called": [], "taken": []}

    def new(shape, dtype, device, stream, returned=True):
        seen["taken"].append(stream)
        return torch.zeros(shape, dtype=dtype).as_subclass(Tensor)

    def empty(dtype, device, stream, *shape):
        return new(shape, dtype, device, stream) if stream is None else real(dtype, device, stream, *shape)

    def launch(f, device, stream, *args):
        assert device == 0
        seen["called"].append((f.__name__, stream))

    real = tw._empty
    monkeypatch.setattr(tw, "_new", new)
    monkeypatch.setattr(tw, "_empty", empty)
    monkeypatch.setattr(tw, "_launch", launch)
    return seen


def test_launches_on_the_device_and_stream_asked_for(monkeypatch):
    """On the current device and stream at once, on others through _call."""
    seen = []

    def f(*args):
        seen.append(args)
        return 0

    monkeypatch.setattr(tw, "_torch", types.SimpleNamespace(_C=types.SimpleNamespace(_cuda_getDevice=lambda: 1)))
    monkeypatch.setattr(tw, "_raw_stream", lambda device: 70 + device)
    monkeypatch.setattr(tw, "_call", lambda *a: seen.append(a))
    tw._launch(f, 1, None, 5)
    tw._launch(f, 0, None, 5)
    tw._launch(f, 1, "side", 5)
    assert seen == [(5, 71), ("f", 0, None, 5), ("f", 1, "side", 5)]
    monkeypatch.setattr(tw, "_check", lambda name, rc: seen.append((name, rc)))
    tw._launch(lambda *a: 3, 1, None)
    assert seen[-1] == ("<lambda>", 3)


def batch(nseq=2, width=3):
    return tw.I8KvBatch(fake(nseq + 1), fake(nseq), fake(nseq, width))


def cache(blocks=4, heads=2, d=64):
    return tw.I8KvCache(codes=fake(blocks, heads, 2, 64 * d, dtype=torch.int8),
                        scales=fake(blocks, heads, 2, dtype=torch.float32))


N, K = 20, 256
f16 = torch.float16
CALLS = {
    "q4_pack": lambda s, **kw: tw.q4_pack(kw.get("t", fake(N, K, dtype=torch.int8)),
                                          kw.get("scale", fake(N, K // 32, dtype=f16)), stream=s, out=kw.get("out")),
    "q4_gemv": lambda s, **kw: tw.q4_gemv(kw.get("packed", fake(32 * K // 2 + 32 * K // 16, dtype=torch.uint8)), N, K, 32,
                                          kw.get("x", fake(3, K, dtype=torch.bfloat16)), y=kw.get("y"), stream=s),
    "q4_gemv_i8": lambda s, **kw: tw.q4_gemv_i8(fake(32 * K // 2 + 32 * K // 16, dtype=torch.uint8), N, K, 32,
                                                kw.get("q", fake(3, K, dtype=torch.int8)),
                                                kw.get("s_x", fake(3, dtype=torch.float32)), y=kw.get("y"), stream=s),
    "draft_tree_mask": lambda s, **kw: tw.draft_tree_mask(batch(), kw.get("parent", fake(5)), kw.get("words", 1),
                                                          mask=kw.get("mask"), pos=kw.get("pos"), stream=s),
    "i8_kv_attend_tree": lambda s, **kw: tw.i8_kv_attend_tree(
        cache(), batch(width=800), kw.get("q", fake(5, 4, 64, dtype=torch.bfloat16)),
        kw.get("mask", fake(5, 1, dtype=torch.int64)), out=kw.get("out"), workspace=kw.get("workspace"), stream=s),
    "draft_tree_accept": lambda s, **kw: tw.draft_tree_accept(
        batch(), fake(5), kw.get("token", fake(5)), kw.get("target", fake(5)), 4, path=kw.get("path"),
        count=kw.get("count"), following=kw.get("following"), stream=s),
    "i8_kv_keep": lambda s, **kw: tw.i8_kv_keep(cache(), kw.get("batch", batch()), 5, kw.get("path", fake(2, 4)),
                                                lens_out=kw.get("lens_out"), stream=s),
}


def test_every_call_with_a_stream_is_here():
    takes = {n for m in HELD for n, f in vars(m).items() if inspect.isfunction(f) and not n.startswith("_")
             and "stream" in inspect.signature(f).parameters}
    assert takes == set(CALLS)


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_given_stream(calls, name):
    side = object()
    CALLS[name](side)
    assert calls["called"] == [(name, side)]
    assert calls["taken"] and all(s is side for s in calls["taken"])


@pytest.mark.parametrize("name, kw, message", [
    ("q4_pack", dict(t=fake(N, K)), "dtype"),
    ("q4_pack", dict(scale=fake(N + 1, K // 32, dtype=f16)), "scale has shape"),
    ("q4_pack", dict(scale=fake(N, 7, dtype=f16)), "scale has shape"),
    ("q4_pack", dict(scale=fake(N, 1, dtype=f16)), "invalid shape"),
    ("q4_pack", dict(out=fake(3, dtype=torch.uint8)), "at least"),
    ("q4_gemv", dict(x=fake(3, K + 128, dtype=torch.bfloat16)), "expected contiguous"),
    ("q4_gemv", dict(x=fake(3, K)), "dtype"),
    ("q4_gemv", dict(x=fake(3, 2 * K, dtype=torch.bfloat16)[:, ::2]), "expected contiguous"),
    ("q4_gemv", dict(packed=fake(32 * K // 2, dtype=torch.uint8)), "at least"),
    ("q4_gemv", dict(y=fake(N, 3, dtype=torch.float32)), "shape"),
    ("q4_gemv_i8", dict(s_x=fake(2, dtype=torch.float32)), "shape"),
    ("q4_gemv_i8", dict(q=fake(3, K, dtype=torch.uint8)), "dtype"),
    ("draft_tree_mask", dict(words=0), "words"),
    ("draft_tree_mask", dict(words=9), "words"),
    ("draft_tree_mask", dict(parent=fake(5, dtype=torch.int64)), "dtype"),
    ("draft_tree_mask", dict(mask=fake(5, 2, dtype=torch.int64)), "shape"),
    ("draft_tree_mask", dict(pos=fake(4)), "shape"),
    ("i8_kv_attend_tree", dict(mask=fake(4, 1, dtype=torch.int64)), "shape"),
    ("i8_kv_attend_tree", dict(mask=fake(5, 1)), "dtype"),
    ("i8_kv_attend_tree", dict(q=fake(5, 4, 128, dtype=torch.bfloat16)), "shape"),
    ("i8_kv_attend_tree", dict(out=fake(5, 4, 64)), "dtype"),
    ("i8_kv_attend_tree", dict(workspace=fake(1)), "workspace"),
    ("draft_tree_accept", dict(token=fake(6)), "shape"),
    ("draft_tree_accept", dict(path=fake(2, 3)), "shape"),
    ("draft_tree_accept", dict(count=fake(3)), "shape"),
    ("i8_kv_keep", dict(path=fake(3, 4)), "shape"),
    ("i8_kv_keep", dict(path=fake(2, 8)[:, ::2]), "contiguous"),
    ("i8_kv_keep", dict(lens_out=fake(3)), "shape"),
])
def test_refused(calls, name, kw, message):
    with pytest.raises(RuntimeError, match=message):
        CALLS[name](None, **kw)
    assert not calls["called"]


def test_lens_out_may_not_be_lens(calls):
    b = batch()
    with pytest.raises(RuntimeError, match="lens_out"):
        CALLS["i8_kv_keep"](None, batch=b, lens_out=b.lens)
    n = b.nseq
    lengths = fake(3 * n)
    b.lens = lengths[n:2 * n]
    for start in (1, n + 1, 2 * n - 1):          # in part the same memory
        with pytest.raises(RuntimeError, match="lens_out"):
            CALLS["i8_kv_keep"](None, batch=b, lens_out=lengths[start:start + n])
    assert n > 1 and not calls["called"]
    for start in (0, 2 * n):                     # side by side
        CALLS["i8_kv_keep"](None, batch=b, lens_out=lengths[start:start + n])
    assert len(calls["called"]) == 2


def test_another_device_is_refused(calls):
    b = batch()
    b.device = 1
    with pytest.raises(RuntimeError, match="device"):
        CALLS["i8_kv_keep"](None, batch=b)


def test_a_workspace_for_every_smaller_batch(monkeypatch):
    """What a server sizes once for its largest batch, which needs none itself."""
    monkeypatch.setattr(draft_tree._torch, "empty", lambda n, dtype, device: torch.zeros(n, dtype=dtype))
    c = types.SimpleNamespace(heads=8, d=128, device=0)
    large = types.SimpleNamespace(nseq=100, width=250)
    assert tw.i8_kv_attend_tree_workspace_bytes(2400, 32, 8, 128, 100, 16000) == 0
    for max_len in (None, 16000):
        ws = tw.i8_kv_attend_tree_workspace(c, large, 2400, 32, max_len)
        assert ws.nbytes >= max(tw.i8_kv_attend_tree_workspace_bytes(24 * n, 32, 8, 128, n, m)
                                for n in range(1, 101) for m in (500, 4000, 16000, 10 ** 6))
    assert tw.i8_kv_attend_tree_workspace(c, large, 0, 32) is None
    for kw in (dict(tokens=-1), dict(hq=3), dict(max_len=0), dict(max_len=2 ** 31)):
        with pytest.raises(RuntimeError):
            tw.i8_kv_attend_tree_workspace(c, large, **{**dict(tokens=8, hq=32), **kw})
