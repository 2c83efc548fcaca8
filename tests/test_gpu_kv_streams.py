"""Calls on the current stream and on another one, one right after the other."""
import pytest

import ternary_weight_decode_amd as tw

from test_gpu_kv import Case, dev, queries

pytestmark = pytest.mark.gpu


def cases():
    import torch
    out = []
    for i in range(4):
        s = Case(tw, 400 + i, 128, 2, [1, 2], [5000 + 900 * i, 3000])
        out.append((*s.device(), dev(queries(s, 8), torch.bfloat16), s))
    return out


def test_attend_on_the_current_stream_then_on_another():
    """Workspaces are dropped as each call returns, with its kernels still to run; the next call, on
    another stream, may not be given the same bytes."""
    import torch
    parts = cases()
    c, b, q, s = parts[0]
    assert tw.i8_kv_attend_workspace(c, b, s.tokens, 8) is not None
    want = [tw.i8_kv_attend(c, b, q) for c, b, q, _ in parts]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        got = [tw.i8_kv_attend(c, b, q, stream=side if i % 2 else None) for i, (c, b, q, _) in enumerate(parts)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_outputs_dropped_on_one_stream_are_not_written_by_another():
    import torch
    parts = cases()
    f = tw.QkTransform(128)
    rows = [dev(s.rng.normal(size=(3000, 10, 128)).astype("float32")) for *_, s in parts]
    want = [tw.qk_norm_rope(f, r, None)[0] for r in rows]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        kept = []
        for i, r in enumerate(rows):
            tw.qk_norm_rope(f, rows[i - 1], None)                   # dropped at once, on the current stream
            kept.append(tw.qk_norm_rope(f, r, None, stream=side)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, want))
