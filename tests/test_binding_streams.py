"""Every call of the binding that allocates takes the memory from the stream
that it is given (no GPU: the library and the allocator are stood in for)."""
import inspect

import pytest
import torch

import ternary_weight_decode_amd as tw

N, K, M, V, B = 64, 512, 2, 48, 2
i8 = lambda *s: torch.zeros(s, dtype=torch.int8)
f32 = lambda *s: torch.zeros(s)
b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
blob = torch.zeros(8, dtype=torch.uint8)
ids = torch.zeros(M, dtype=torch.int32)

CALLS = {
    "tern_pack": lambda s: tw.tern_pack(i8(N, K), torch.zeros(N, K // 128, dtype=torch.float16), stream=s),
    "tern_stats": lambda s: tw.tern_stats(blob, N, K, stream=s),
    "tern_quantize_i8": lambda s: tw.tern_quantize_i8(b16(M, K), stream=s),
    "tern_gemv": lambda s: tw.tern_gemv(blob, N, K, b16(M, K), stream=s),
    "tern_gemv_i8": lambda s: tw.tern_gemv_i8(blob, N, K, i8(M, K), f32(M), stream=s),
    "i8_head_gemv": lambda s: tw.i8_head_gemv(i8(V, K), f32(V), b16(M, K), stream=s),
    "i8_head_gemv_i8": lambda s: tw.i8_head_gemv_i8(i8(V, K), f32(V), i8(M, K), f32(M), stream=s),
    "i8_head_pack": lambda s: tw.i8_head_pack(i8(V, K), stream=s),
    "i8_head_gemv_packed": lambda s: tw.i8_head_gemv_packed(blob, f32(V), V, K, b16(M, K), stream=s),
    "i8_head_gemv_packed_i8": lambda s: tw.i8_head_gemv_packed_i8(blob, f32(V), V, K, i8(M, K), f32(M), stream=s),
    "i8_head_argmax_packed": lambda s: tw.i8_head_argmax_packed(blob, f32(V), V, K, b16(M, K), stream=s),
    "i8_head_argmax_packed_i8": lambda s: tw.i8_head_argmax_packed_i8(blob, f32(V), V, K, i8(M, K), f32(M), stream=s),
    "i8_head_argmax": lambda s: tw.i8_head_argmax(i8(V, K), f32(V), b16(M, K), stream=s),
    "i8_head_argmax_i8": lambda s: tw.i8_head_argmax_i8(i8(V, K), f32(V), i8(M, K), f32(M), stream=s),
    "tern_gemm_prefill": lambda s: tw.tern_gemm_prefill(blob, N, K, i8(M, K), f32(M), stream=s),
    "tern5_pack": lambda s: tw.tern5_pack(i8(N, K), f32(N, B), f32(N, B), stream=s),
    "tern5_gemv": lambda s: tw.tern5_gemv(blob, N, K, b16(M, K), stream=s),
    "tern5_gemv_i8": lambda s: tw.tern5_gemv_i8(blob, N, K, i8(M, K), f32(M), stream=s),
    "fv5b_head_gemv": lambda s: tw.fv5b_head_gemv(i8(V, K), f32(V, B), b16(M, K), stream=s),
    "fv5b_head_gemv_i8": lambda s: tw.fv5b_head_gemv_i8(i8(V, K), f32(V, B), i8(M, K), f32(M), stream=s),
    "fv5b_head_argmax": lambda s: tw.fv5b_head_argmax(i8(V, K), f32(V, B), b16(M, K), stream=s),
    "fv5b_head_argmax_i8": lambda s: tw.fv5b_head_argmax_i8(i8(V, K), f32(V, B), i8(M, K), f32(M), stream=s),
    "fv5b_head_gemv_packed": lambda s: tw.fv5b_head_gemv_packed(blob, f32(V, B), V, K, b16(M, K), stream=s),
    "fv5b_head_gemv_packed_i8":
        lambda s: tw.fv5b_head_gemv_packed_i8(blob, f32(V, B), V, K, i8(M, K), f32(M), stream=s),
    "fv5b_head_argmax_packed": lambda s: tw.fv5b_head_argmax_packed(blob, f32(V, B), V, K, b16(M, K), stream=s),
    "fv5b_head_argmax_packed_i8":
        lambda s: tw.fv5b_head_argmax_packed_i8(blob, f32(V, B), V, K, i8(M, K), f32(M), stream=s),
    "fv5b_head_argmax_embed": lambda s: tw.fv5b_head_argmax_embed(i8(V, K), f32(V, B), b16(M, K), i8(V, K), f32(V, B),
                                                                 stream=s),
    "fv5b_embed": lambda s: tw.fv5b_embed(i8(V, K), f32(V, B), ids, stream=s),
    "tern_launch_probe": lambda s: tw.tern_launch_probe("store", 4, stream=s),
    "tern_mfma_peak": lambda s: tw.tern_mfma_peak("int8", 1, 4, stream=s),
}
# given what they write, or tested in test_kv_binding.py
OTHERS = {"i8_head_argmax_noalloc", "tern_chain_plan", "tern_gemv_chain", "qk_norm_rope", "i8_kv_append", "i8_kv_read",
          "i8_kv_attend"}


class Library:
    """Status functions do nothing; sizes are the library's own."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        return (lambda *a: 0) if name in tw._INT_STATUS else getattr(self.real, name)


def test_every_call_with_a_stream_is_here():
    takes = {n for n, f in vars(tw).items() if inspect.isfunction(f) and not n.startswith("_")
             and "stream" in inspect.signature(f).parameters}
    assert takes == set(CALLS) | OTHERS


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_given_stream(monkeypatch, name):
    library, taken = Library(tw.lib()), []

    def new(shape, dtype, device, stream, returned=True):
        taken.append(stream)
        return torch.zeros(shape, dtype=dtype)

    def empty(*a, **k):
        raise AssertionError("allocated on whatever stream is current")

    side = object()
    monkeypatch.setattr(tw, "lib", lambda: library)
    monkeypatch.setattr(tw, "_need", lambda *a: None)
    monkeypatch.setattr(tw, "_stream", lambda stream: stream)
    monkeypatch.setattr(tw, "_new", new)
    monkeypatch.setattr(torch, "empty", empty)
    CALLS[name](side)
    assert taken and all(s is side for s in taken)
