"""The cache calls refuse a stream of another device than their tensors' (no GPU)."""
import types

import pytest

import ternary_weight_decode_amd as tw


def test_a_stream_of_another_device_is_refused(monkeypatch):
    called = []
    monkeypatch.setattr(tw, "_torch", types.SimpleNamespace(cuda=types.SimpleNamespace(current_device=lambda: 0)))
    monkeypatch.setattr(tw, "_lib", types.SimpleNamespace(i8_kv_read=lambda *a: called.append(a) or 0))
    stream = types.SimpleNamespace(device_index=1, cuda_stream=7)
    with pytest.raises(RuntimeError, match="stream is on device 1, expected 0"):
        tw._call("i8_kv_read", 0, stream)
    assert called == []
    stream.device_index = 0
    tw._call("i8_kv_read", 0, stream)
    assert called == [(7,)]
