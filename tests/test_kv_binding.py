"""Host side of the cache calls' binding, with torch and the library stood in for (no GPU)."""
import contextlib
import types

import pytest

import ternary_weight_decode_amd as tw


class Memory:
    def __init__(self, stream):
        self.allocated_on, self.recorded = stream, []

    def record_stream(self, stream):
        self.recorded.append(stream)


class Torch:
    """Streams by name; the one in use when `empty` is called is the one whose memory it hands out."""

    def __init__(self, monkeypatch):
        self.current = "current"
        self.cuda = types.SimpleNamespace(current_stream=lambda device: self.current, stream=self.use)
        monkeypatch.setattr(tw, "_torch", self)

    @contextlib.contextmanager
    def use(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before

    def empty(self, shape, dtype, device):
        return Memory(self.current)


@pytest.mark.parametrize("stream, used", [(None, "current"), ("current", "current"), ("side", "side")])
def test_memory_comes_from_the_stream_that_uses_it(monkeypatch, stream, used):
    torch = Torch(monkeypatch)
    out = tw._new((1,), "uint8", 0, stream)
    assert out.allocated_on == used and torch.current == "current"
    # whoever gets it back uses it on the stream that was current
    assert out.recorded == ([] if used == "current" else ["current"])


def test_a_workspace_stays_with_its_stream(monkeypatch):
    Torch(monkeypatch)
    ws = tw._new(5, "uint8", 0, "side", returned=False)
    assert ws.allocated_on == "side" and ws.recorded == []
