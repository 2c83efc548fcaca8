"""Python binding of libtern.so — gfx950 ternary-weight GEMV / GEMM kernels.

Thin argument marshalling over the C ABI of ``include/tern.h``: every call
takes torch tensors that already live on the GPU, passes their device
pointers and the current HIP stream to the library, and raises
``RuntimeError`` with the library's status text on any error.  torch is used
for device memory and streams only; every step of the computation runs in the
library's HIP kernels.  There is no fallback: if ``libtern.so`` is missing or
fails to load, every call raises.

Names follow the C ABI: ``tern_pack``, ``tern_stats``, ``tern_quantize_i8``,
``tern_gemv``, ``tern_gemv_i8``, ``i8_head_gemv``, ``i8_head_gemv_i8``,
``tern_gemm_prefill``, ``tern_packed_bytes``, and the dependent-GEMV chain
``tern_chain_workspace_bytes``, ``tern_chain_plan``, ``tern_gemv_chain``, the
fused head + greedy argmax ``i8_head_argmax[_i8]``, and the five-level
(FV5-style) weights ``tern5_packed_bytes``, ``tern5_pack``, ``tern5_gemv[_i8]``, and the
block-scaled int8 head and embedding (FV5B-style) ``fv5b_head_gemv[_i8]``,
``fv5b_head_argmax[_i8]``, ``fv5b_head_argmax_embed``, ``fv5b_embed`` (and
``fv5b_head_gemv_packed[_i8]``, ``fv5b_head_argmax_packed[_i8]`` over the
packed copy), the
packed int8 head ``i8_head_packed_bytes``, ``i8_head_pack``,
``i8_head_gemv_packed[_i8]``, ``i8_head_argmax_packed[_i8]``, the attention
side of a step ``qk_norm_rope``, ``i8_kv_append``, ``i8_kv_read`` and
``i8_kv_attend`` (with the handles ``QkTransform``, ``I8KvCache`` and
``I8KvBatch``), and the launch-configuration views
``tern_gemv_config``, ``tern_prefill_config`` and ``i8_kv_attend_config``.
"""
from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtern.so")
MAX_M_GEMV = 16
SYMBOLS = ("tern_strerror", "tern_last_error", "tern_abi_version", "tern_packed_bytes", "tern_pack", "tern_stats",
           "tern_quantize_i8", "tern_gemv", "tern_gemv_i8", "i8_head_gemv", "i8_head_gemv_i8", "tern_gemm_prefill",
           "tern_chain_workspace_bytes", "tern_chain_plan", "tern_gemv_chain", "i8_head_argmax_workspace_bytes",
           "i8_head_argmax", "i8_head_argmax_i8", "tern5_packed_bytes", "tern5_pack", "tern5_gemv", "tern5_gemv_i8",
           "fv5b_head_gemv", "fv5b_head_gemv_i8", "fv5b_head_argmax", "fv5b_head_argmax_i8", "fv5b_head_argmax_embed", "fv5b_embed",
           "tern_gemv_config", "tern_prefill_config", "tern_mfma_peak_ops", "tern_mfma_peak_sink_bytes", "tern_mfma_peak",
           "tern_launch_probe", "i8_head_argmax_noalloc", "i8_head_packed_bytes", "i8_head_pack",
           "i8_head_gemv_packed", "i8_head_gemv_packed_i8", "i8_head_argmax_packed", "i8_head_argmax_packed_i8",
           "fv5b_head_gemv_packed", "fv5b_head_gemv_packed_i8", "fv5b_head_argmax_packed",
           "fv5b_head_argmax_packed_i8", "qk_norm_rope", "i8_kv_append", "i8_kv_read",
           "i8_kv_attend_workspace_bytes", "i8_kv_attend", "i8_kv_attend_config")
_INT_STATUS = ("tern_pack", "tern_stats", "tern_quantize_i8", "tern_gemv", "tern_gemv_i8", "i8_head_gemv",
               "i8_head_gemv_i8", "tern_gemm_prefill", "tern_chain_plan", "tern_gemv_chain", "i8_head_argmax",
               "i8_head_argmax_i8", "tern5_pack", "tern5_gemv", "tern5_gemv_i8", "fv5b_head_gemv", "fv5b_head_gemv_i8",
               "fv5b_head_argmax", "fv5b_head_argmax_i8", "fv5b_head_argmax_embed", "fv5b_embed", "tern_mfma_peak",
               "tern_launch_probe", "i8_head_argmax_noalloc", "i8_head_pack", "i8_head_gemv_packed",
               "i8_head_gemv_packed_i8", "i8_head_argmax_packed", "i8_head_argmax_packed_i8",
               "fv5b_head_gemv_packed", "fv5b_head_gemv_packed_i8", "fv5b_head_argmax_packed",
               "fv5b_head_argmax_packed_i8", "qk_norm_rope", "i8_kv_append", "i8_kv_read", "i8_kv_attend")
KV_BLOCK = 64

_lib = None
_i64 = ctypes.c_int64
_p = ctypes.c_void_p


class TernChainStep(ctypes.Structure):
    """struct tern_chain_step of include/tern.h."""
    _fields_ = [("packed", _p), ("N", _i64), ("K", _i64), ("x", _p), ("x_from", _i64), ("y", _p)]


class _KvCache(ctypes.Structure):
    """struct i8_kv_cache of include/tern.h."""
    _fields_ = [("codes", _p), ("scales", _p), ("blocks", _i64), ("heads", _i64), ("D", _i64)]


class _KvBatch(ctypes.Structure):
    """struct i8_kv_batch of include/tern.h."""
    _fields_ = [("cu", _p), ("lens", _p), ("table", _p), ("nseq", _i64), ("table_width", _i64),
                ("table_stride", _i64)]


class _QkTransform(ctypes.Structure):
    """struct tern_qk_transform of include/tern.h."""
    _fields_ = [("q_gain", _p), ("k_gain", _p), ("inv_freq", _p), ("eps", ctypes.c_float),
                ("interleaved", ctypes.c_int32)]


def lib():
    """Load libtern.so (built in-tree by ternary_weight_decode_amd.build); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m ternary_weight_decode_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.tern_strerror.restype = ctypes.c_char_p
        L.tern_strerror.argtypes = [ctypes.c_int]
        L.tern_last_error.restype = ctypes.c_char_p
        L.tern_abi_version.restype = ctypes.c_int
        L.tern_packed_bytes.restype = _i64
        L.tern_packed_bytes.argtypes = [_i64, _i64]
        L.tern_pack.argtypes = [_p, _p, _i64, _i64, _p, _p]
        L.tern_stats.argtypes = [_p, _i64, _i64, _p, _p]
        L.tern_quantize_i8.argtypes = [_p, _i64, _i64, _p, _p, _p]
        L.tern_gemv.argtypes = [_p, _i64, _i64, _p, _i64, _p, _p]
        L.tern_gemv_i8.argtypes = [_p, _i64, _i64, _p, _p, _i64, _p, _p, _p]
        L.i8_head_gemv.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p]
        L.i8_head_gemv_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p]
        L.tern_gemm_prefill.argtypes = [_p, _i64, _i64, _p, _p, _i64, _p, _p, _p]
        L.tern_chain_workspace_bytes.restype = _i64
        L.tern_chain_workspace_bytes.argtypes = [ctypes.POINTER(TernChainStep), _i64]
        L.tern_chain_plan.argtypes = [ctypes.POINTER(TernChainStep), _i64, _p, _i64, _p]
        L.tern_gemv_chain.argtypes = [_p, _i64, _p]
        L.i8_head_argmax_workspace_bytes.restype = _i64
        L.i8_head_argmax_workspace_bytes.argtypes = [_i64, _i64]
        L.i8_head_argmax.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p]
        L.i8_head_argmax_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p, _p, _p]
        L.i8_head_argmax_noalloc.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p]
        L.tern5_packed_bytes.restype = _i64
        L.tern5_packed_bytes.argtypes = [_i64, _i64]
        L.tern5_pack.argtypes = [_p, _p, _p, _i64, _i64, _p, _p]
        L.tern5_gemv.argtypes = [_p, _i64, _i64, _p, _i64, _p, _p]
        L.tern5_gemv_i8.argtypes = [_p, _i64, _i64, _p, _p, _i64, _p, _p, _p]
        L.fv5b_head_gemv.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p]
        L.fv5b_head_gemv_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p]
        L.fv5b_head_argmax.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p]
        L.fv5b_head_argmax_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p, _p, _p]
        L.fv5b_embed.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p, _p]
        L.fv5b_head_argmax_embed.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p, _p, _i64, _i64, _p, _p,
                                             _p]
        L.tern_gemv_config.restype = ctypes.c_int
        L.tern_gemv_config.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(_i64)]
        L.tern_prefill_config.restype = ctypes.c_int
        L.tern_prefill_config.argtypes = [_i64, _i64, _i64, ctypes.POINTER(_i64)]
        L.tern_mfma_peak_ops.restype = ctypes.c_double
        L.tern_mfma_peak_ops.argtypes = [ctypes.c_int, _i64, _i64]
        L.tern_mfma_peak_sink_bytes.restype = _i64
        L.tern_mfma_peak_sink_bytes.argtypes = [_i64]
        L.tern_mfma_peak.argtypes = [ctypes.c_int, _i64, _i64, _p, _p]
        L.tern_launch_probe.argtypes = [ctypes.c_int, _i64, _p, _i64, _p, _p]
        L.i8_head_packed_bytes.restype = _i64
        L.i8_head_packed_bytes.argtypes = [_i64, _i64]
        L.i8_head_pack.argtypes = [_p, _i64, _i64, _p, _p]
        L.i8_head_gemv_packed.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p]
        L.i8_head_gemv_packed_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p]
        L.i8_head_argmax_packed.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p]
        L.i8_head_argmax_packed_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p, _p, _p]
        L.fv5b_head_gemv_packed.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p]
        L.fv5b_head_gemv_packed_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p]
        L.fv5b_head_argmax_packed.argtypes = [_p, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p]
        L.fv5b_head_argmax_packed_i8.argtypes = [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p, _p, _p]
        L.i8_kv_attend_config.restype = ctypes.c_int
        L.i8_kv_attend_config.argtypes = [_i64] * 9 + [ctypes.POINTER(_i64)]
        cache, batch, transform = (ctypes.POINTER(t) for t in (_KvCache, _KvBatch, _QkTransform))
        L.qk_norm_rope.argtypes = [transform, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, ctypes.c_int, _p, _p, _p,
                                   ctypes.c_int, _p]
        L.i8_kv_append.argtypes = [cache, batch, transform, _i64, _p, _i64, _i64, _p, _i64, _p, _i64, ctypes.c_int,
                                   _p, _p, _p]
        L.i8_kv_read.argtypes = [cache, batch, _i64, _p, _p, ctypes.c_int, _p]
        L.i8_kv_attend_workspace_bytes.restype = _i64
        L.i8_kv_attend_workspace_bytes.argtypes = [_i64] * 7
        L.i8_kv_attend.argtypes = [cache, batch, _i64, _p, _i64, _i64, ctypes.c_float, _i64, _i64, _i64, _p, _p, _p]
        for name in _INT_STATUS:
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(name: str, rc: int):
    if rc != 0:
        L = lib()
        raise RuntimeError(f"{name}: {L.tern_strerror(rc).decode()} {L.tern_last_error().decode()}".strip())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, dtypes, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA/HIP tensor")
    if t.dtype not in dtypes:
        raise RuntimeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise RuntimeError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise RuntimeError(f"{name} must have {ndim} dimensions")


def tern_packed_bytes(n: int, k: int) -> int:
    return int(lib().tern_packed_bytes(n, k))


def tern_pack(t, scale, out=None, stream=None):
    """t int8 [N,K] in {-1,0,1}; scale fp16 bits [N,K/128] (int16/uint16/float16) -> packed uint8 blob."""
    import torch
    _need(t, "t", (torch.int8,), 2)
    _need(scale, "scale", (torch.int16, torch.uint16, torch.float16), 2)
    n, k = t.shape
    nbytes = tern_packed_bytes(n, k)
    if nbytes < 0:
        _check("tern_pack", 2)
    if out is None:
        out = _new(nbytes, torch.uint8, t.device, stream)
    _check("tern_pack", lib().tern_pack(_ptr(t), _ptr(scale), n, k, _ptr(out), _stream(stream)))
    return out


def tern_stats(packed, n: int, k: int, out=None, stream=None):
    """-> int64 [3]: nonzero weights, -1 weights, non-canonical sign bits."""
    import torch
    if out is None:
        out = _new(3, torch.int64, packed.device, stream)
    _check("tern_stats", lib().tern_stats(_ptr(packed), n, k, _ptr(out), _stream(stream)))
    return out


def tern_quantize_i8(x, q=None, s_x=None, stream=None):
    """x bf16 [M,K] -> (q int8 [M,K], s_x fp32 [M])."""
    import torch
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    m, k = x.shape
    if q is None:
        q = _new((m, k), torch.int8, x.device, stream)
    if s_x is None:
        s_x = _new(m, torch.float32, x.device, stream)
    _check("tern_quantize_i8", lib().tern_quantize_i8(_ptr(x), m, k, _ptr(q), _ptr(s_x), _stream(stream)))
    return q, s_x


def tern_gemv(packed, n: int, k: int, x, y=None, stream=None):
    """y[m,n] = sum_b scale[n,b] sum_{k in b} t[n,k] x[m,k]; x bf16 [M,K], M <= 16 -> y fp32 [M,N]."""
    import torch
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    m = x.shape[0]
    if y is None:
        y = _new((m, n), torch.float32, x.device, stream)
    _check("tern_gemv", lib().tern_gemv(_ptr(packed), n, k, _ptr(x), m, _ptr(y), _stream(stream)))
    return y


def tern_gemv_i8(packed, n: int, k: int, q, s_x, y=None, acc=None, stream=None):
    """int8 activations: y = s_x[m] * sum_b scale[n,b] acc[m,n,b]; acc (optional) int32 [M,N,K/128]."""
    import torch
    _need(q, "q", (torch.int8,), 2)
    m = q.shape[0]
    if y is None:
        y = _new((m, n), torch.float32, q.device, stream)
    _check("tern_gemv_i8", lib().tern_gemv_i8(_ptr(packed), n, k, _ptr(q), _ptr(s_x), m, _ptr(y), _ptr(acc),
                                              _stream(stream)))
    return y


def i8_head_gemv(w, row_scale, x, y=None, stream=None):
    """logits[m,v] = row_scale[v] sum_k W[v,k] x[m,k]; W int8 [V,K], x bf16 [M,K]."""
    import torch
    _need(w, "W", (torch.int8,), 2)
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    v, k = w.shape
    m = x.shape[0]
    if y is None:
        y = _new((m, v), torch.float32, x.device, stream)
    _check("i8_head_gemv", lib().i8_head_gemv(_ptr(w), _ptr(row_scale), v, k, _ptr(x), m, _ptr(y),
                                              _stream(stream)))
    return y


def i8_head_gemv_i8(w, row_scale, q, s_x, y=None, acc=None, stream=None):
    import torch
    _need(w, "W", (torch.int8,), 2)
    _need(q, "q", (torch.int8,), 2)
    v, k = w.shape
    m = q.shape[0]
    if y is None:
        y = _new((m, v), torch.float32, q.device, stream)
    _check("i8_head_gemv_i8", lib().i8_head_gemv_i8(_ptr(w), _ptr(row_scale), v, k, _ptr(q), _ptr(s_x), m, _ptr(y),
                                                    _ptr(acc), _stream(stream)))
    return y


def i8_head_packed_bytes(v: int, k: int) -> int:
    return int(lib().i8_head_packed_bytes(v, k))


def i8_head_pack(w, out=None, stream=None):
    """W int8 [V,K] -> its packed copy (int8, i8_head_packed_bytes(V, K) bytes) for i8_head_gemv_packed[_i8]."""
    import torch
    _need(w, "W", (torch.int8,), 2)
    v, k = w.shape
    nbytes = i8_head_packed_bytes(v, k)
    if nbytes < 0:
        _check("i8_head_pack", 2)
    if out is None:
        out = _new(nbytes, torch.int8, w.device, stream)
    _check("i8_head_pack", lib().i8_head_pack(_ptr(w), v, k, _ptr(out), _stream(stream)))
    return out


def i8_head_gemv_packed(wp, row_scale, v: int, k: int, x, y=None, stream=None):
    """i8_head_gemv over the packed copy wp of W [v,k]; x bf16 [M,K] -> logits fp32 [M,V]."""
    import torch
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    m = x.shape[0]
    if y is None:
        y = _new((m, v), torch.float32, x.device, stream)
    _check("i8_head_gemv_packed", lib().i8_head_gemv_packed(_ptr(wp), _ptr(row_scale), v, k, _ptr(x), m, _ptr(y),
                                                            _stream(stream)))
    return y


def i8_head_gemv_packed_i8(wp, row_scale, v: int, k: int, q, s_x, y=None, acc=None, stream=None):
    import torch
    _need(q, "q", (torch.int8,), 2)
    m = q.shape[0]
    if y is None:
        y = _new((m, v), torch.float32, q.device, stream)
    _check("i8_head_gemv_packed_i8", lib().i8_head_gemv_packed_i8(_ptr(wp), _ptr(row_scale), v, k, _ptr(q),
                                                                  _ptr(s_x), m, _ptr(y), _ptr(acc), _stream(stream)))
    return y


def i8_head_argmax_packed(wp, row_scale, v: int, k: int, x, workspace=None, logits=None, stream=None):
    """i8_head_argmax over the packed copy wp of W [v,k]: (idx int32 [M], val fp32 [M])."""
    import torch
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    m = x.shape[0]
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, x.device, stream, returned=False)
    idx = _new(m, torch.int32, x.device, stream)
    val = _new(m, torch.float32, x.device, stream)
    _check("i8_head_argmax_packed", lib().i8_head_argmax_packed(_ptr(wp), _ptr(row_scale), v, k, _ptr(x), m,
                                                                _ptr(idx), _ptr(val), _ptr(logits),
                                                                _ptr(workspace), _stream(stream)))
    return idx, val


def i8_head_argmax_packed_i8(wp, row_scale, v: int, k: int, q, s_x, workspace=None, logits=None, stream=None):
    import torch
    _need(q, "q", (torch.int8,), 2)
    m = q.shape[0]
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, q.device, stream, returned=False)
    idx = _new(m, torch.int32, q.device, stream)
    val = _new(m, torch.float32, q.device, stream)
    _check("i8_head_argmax_packed_i8", lib().i8_head_argmax_packed_i8(_ptr(wp), _ptr(row_scale), v, k, _ptr(q),
                                                                      _ptr(s_x), m, _ptr(idx), _ptr(val),
                                                                      _ptr(logits), _ptr(workspace),
                                                                      _stream(stream)))
    return idx, val


def i8_head_argmax_workspace_bytes(v: int, m: int) -> int:
    return int(lib().i8_head_argmax_workspace_bytes(v, m))


def i8_head_argmax_workspace(v: int, m: int, device="cuda"):
    """A workspace for i8_head_argmax[_i8] over V head rows and up to m activation rows."""
    import torch
    return torch.empty(i8_head_argmax_workspace_bytes(v, m), dtype=torch.uint8, device=device)


def i8_head_argmax(w, row_scale, x, workspace=None, logits=None, stream=None):
    """Greedy argmax over the head logits of bf16 x: (idx int32 [M], val fp32 [M]); logits [M, V] filled when given."""
    import torch
    _need(w, "W", (torch.int8,), 2)
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    v, k = w.shape
    m = x.shape[0]
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, x.device, stream, returned=False)
    idx = _new(m, torch.int32, x.device, stream)
    val = _new(m, torch.float32, x.device, stream)
    _check("i8_head_argmax", lib().i8_head_argmax(_ptr(w), _ptr(row_scale), v, k, _ptr(x), m, _ptr(idx), _ptr(val),
                                                  _ptr(logits), _ptr(workspace), _stream(stream)))
    return idx, val


def i8_head_argmax_noalloc(w, row_scale, x, idx, val, logits=None, stream=None):
    """i8_head_argmax with the keys in the library's own device array: allocates nothing, so the
    caller passes idx (int32 [M]) and val (fp32 [M]); calls overlapping on one device race."""
    import torch
    _need(w, "W", (torch.int8,), 2)
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    v, k = w.shape
    m = x.shape[0]
    _check("i8_head_argmax_noalloc", lib().i8_head_argmax_noalloc(_ptr(w), _ptr(row_scale), v, k, _ptr(x), m,
                                                                  _ptr(idx), _ptr(val), _ptr(logits),
                                                                  _stream(stream)))
    return idx, val


def i8_head_argmax_i8(w, row_scale, q, s_x, workspace=None, logits=None, stream=None):
    """Greedy argmax over the head logits of int8 q (row scales s_x): (idx, val)."""
    import torch
    _need(w, "W", (torch.int8,), 2)
    _need(q, "q", (torch.int8,), 2)
    v, k = w.shape
    m = q.shape[0]
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, q.device, stream, returned=False)
    idx = _new(m, torch.int32, q.device, stream)
    val = _new(m, torch.float32, q.device, stream)
    _check("i8_head_argmax_i8", lib().i8_head_argmax_i8(_ptr(w), _ptr(row_scale), v, k, _ptr(q), _ptr(s_x), m,
                                                        _ptr(idx), _ptr(val), _ptr(logits), _ptr(workspace),
                                                        _stream(stream)))
    return idx, val


def tern_gemm_prefill(packed, n: int, k: int, q, s_x, y=None, acc=None, stream=None):
    import torch
    _need(q, "q", (torch.int8,), 2)
    m = q.shape[0]
    if y is None:
        y = _new((m, n), torch.float32, q.device, stream)
    _check("tern_gemm_prefill", lib().tern_gemm_prefill(_ptr(packed), n, k, _ptr(q), _ptr(s_x), m, _ptr(y),
                                                        _ptr(acc), _stream(stream)))
    return y


def _chain_array(steps):
    """ctypes tern_chain_step array from (packed, N, K, x or None, x_from, y) tuples of tensors."""
    import torch
    arr = (TernChainStep * max(1, len(steps)))()
    for i, (packed, n, k, x, x_from, y) in enumerate(steps):
        _need(packed, "packed", (torch.uint8,))
        _need(y, "y", (torch.float32,))
        if y.numel() != n:
            raise RuntimeError(f"tern_chain: step {i} y has {y.numel()} elements, N = {n}")
        if x is not None:
            _need(x, "x", (torch.int16, torch.uint16, torch.bfloat16))
            if x.numel() != k:
                raise RuntimeError(f"tern_chain: step {i} x has {x.numel()} elements, K = {k}")
        arr[i] = TernChainStep(packed.data_ptr(), n, k, None if x is None else x.data_ptr(), x_from, y.data_ptr())
    return arr


def tern_chain_workspace_bytes(steps) -> int:
    return int(lib().tern_chain_workspace_bytes(_chain_array(steps), len(steps)))


def tern_chain_workspace(steps, device="cuda"):
    """A zero-filled workspace sized for this chain."""
    import torch
    nbytes = tern_chain_workspace_bytes(steps)
    if nbytes < 0:
        _check("tern_chain_workspace_bytes", 2)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def tern_chain_plan(steps, workspace, stream=None):
    """steps: sequence of (packed, N, K, x, x_from, y): x bf16 bits [K] (None when
    x_from >= 0), x_from -1 or an earlier step whose first K outputs, rounded
    to bf16, are x; y fp32 [N].  Writes the device plan into workspace."""
    import torch
    arr = _chain_array(steps)
    _need(workspace, "workspace", (torch.uint8,), 1)
    _check("tern_chain_plan", lib().tern_chain_plan(arr, len(steps), _ptr(workspace), workspace.numel(),
                                                    _stream(stream)))


def tern_gemv_chain(workspace, nsteps: int, stream=None):
    import torch
    _need(workspace, "workspace", (torch.uint8,), 1)
    _check("tern_gemv_chain", lib().tern_gemv_chain(_ptr(workspace), nsteps, _stream(stream)))


def tern_chain_errors(workspace) -> int:
    """Count of aborted waits recorded in a chain workspace (0 in normal operation)."""
    import torch
    return int(workspace[8:12].view(torch.int32).item())


# ---------------------------------------------------------------- five-level

def tern5_packed_bytes(n: int, k: int) -> int:
    return int(lib().tern5_packed_bytes(n, k))


def tern5_pack(levels, s_lo, s_hi, out=None, stream=None):
    """levels int8 [N,K] in [-2,2], K % 512 == 0; s_lo, s_hi fp32 [N,K/256] -> five-level uint8 blob."""
    import torch
    _need(levels, "levels", (torch.int8,), 2)
    _need(s_lo, "s_lo", (torch.float32,), 2)
    _need(s_hi, "s_hi", (torch.float32,), 2)
    n, k = levels.shape
    if tuple(s_lo.shape) != (n, k // 256) or tuple(s_hi.shape) != (n, k // 256):
        raise RuntimeError("tern5_pack: s_lo and s_hi must be [N, K/256]")
    nbytes = tern5_packed_bytes(n, k)
    if nbytes < 0:
        _check("tern5_pack", 2)
    if out is None:
        out = _new(nbytes, torch.uint8, levels.device, stream)
    _check("tern5_pack", lib().tern5_pack(_ptr(levels), _ptr(s_lo), _ptr(s_hi), n, k, _ptr(out), _stream(stream)))
    return out


def tern5_gemv(packed, n: int, k: int, x, y=None, stream=None):
    """y[m,n] = sum_k W[n,k] x[m,k] for the five-level W; x bf16 [M,K], M <= 16 -> y fp32 [M,N]."""
    import torch
    _need(x, "x", (torch.bfloat16, torch.int16, torch.uint16), 2)
    m = x.shape[0]
    if y is None:
        y = _new((m, n), torch.float32, x.device, stream)
    _check("tern5_gemv", lib().tern5_gemv(_ptr(packed), n, k, _ptr(x), m, _ptr(y), _stream(stream)))
    return y


def tern5_gemv_i8(packed, n: int, k: int, q, s_x, y=None, acc=None, stream=None):
    """int8 activations for the five-level W: y = s_x[m] sum_b (s_lo acc_lo + s_hi acc_hi);
    acc (optional) int32 [M,N,K/256,2]."""
    import torch
    _need(q, "q", (torch.int8,), 2)
    m = q.shape[0]
    if y is None:
        y = _new((m, n), torch.float32, q.device, stream)
    _check("tern5_gemv_i8", lib().tern5_gemv_i8(_ptr(packed), n, k, _ptr(q), _ptr(s_x), m, _ptr(y), _ptr(acc),
                                                _stream(stream)))
    return y


# ------------------------------------------------- block-scaled int8 (FV5B)

def _fv5b_args(w, s, act, act_dtypes):
    import torch
    _need(w, "W", (torch.int8,), 2)
    _need(s, "S", (torch.float32,), 2)
    _need(act, "activations", act_dtypes, 2)
    v, k = w.shape
    if tuple(s.shape) != (v, k // 256):
        raise RuntimeError("S must be [V, K/256]")
    return v, k, act.shape[0]


def fv5b_head_gemv(w, s, x, y=None, stream=None):
    """logits[m,v] = sum_b S[v,b] sum_{k in b} W[v,k] x[m,k]; W int8 [V,K], S fp32 [V,K/256], x bf16 [M,K]."""
    import torch
    v, k, m = _fv5b_args(w, s, x, (torch.bfloat16, torch.int16, torch.uint16))
    if y is None:
        y = _new((m, v), torch.float32, x.device, stream)
    _check("fv5b_head_gemv", lib().fv5b_head_gemv(_ptr(w), _ptr(s), v, k, _ptr(x), m, _ptr(y), _stream(stream)))
    return y


def fv5b_head_gemv_i8(w, s, q, s_x, y=None, acc=None, stream=None):
    """int8 activations: logits = s_x[m] sum_b S[v,b] acc[m,v,b]; acc (optional) int32 [M,V,K/256]."""
    import torch
    v, k, m = _fv5b_args(w, s, q, (torch.int8,))
    if y is None:
        y = _new((m, v), torch.float32, q.device, stream)
    _check("fv5b_head_gemv_i8", lib().fv5b_head_gemv_i8(_ptr(w), _ptr(s), v, k, _ptr(q), _ptr(s_x), m, _ptr(y),
                                                        _ptr(acc), _stream(stream)))
    return y


def fv5b_head_argmax(w, s, x, workspace=None, logits=None, stream=None):
    """Greedy argmax over the block-scaled head's logits of bf16 x: (idx int32 [M], val fp32 [M])."""
    import torch
    v, k, m = _fv5b_args(w, s, x, (torch.bfloat16, torch.int16, torch.uint16))
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, x.device, stream, returned=False)
    idx = _new(m, torch.int32, x.device, stream)
    val = _new(m, torch.float32, x.device, stream)
    _check("fv5b_head_argmax", lib().fv5b_head_argmax(_ptr(w), _ptr(s), v, k, _ptr(x), m, _ptr(idx), _ptr(val),
                                                      _ptr(logits), _ptr(workspace), _stream(stream)))
    return idx, val


def fv5b_head_argmax_i8(w, s, q, s_x, workspace=None, logits=None, stream=None):
    """Greedy argmax over the block-scaled head's logits of int8 q: (idx, val)."""
    import torch
    v, k, m = _fv5b_args(w, s, q, (torch.int8,))
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, q.device, stream, returned=False)
    idx = _new(m, torch.int32, q.device, stream)
    val = _new(m, torch.float32, q.device, stream)
    _check("fv5b_head_argmax_i8", lib().fv5b_head_argmax_i8(_ptr(w), _ptr(s), v, k, _ptr(q), _ptr(s_x), m,
                                                            _ptr(idx), _ptr(val), _ptr(logits), _ptr(workspace),
                                                            _stream(stream)))
    return idx, val


def _fv5b_packed_args(s, v, k, act, act_dtypes):
    import torch
    _need(s, "S", (torch.float32,), 2)
    _need(act, "activations", act_dtypes, 2)
    if tuple(s.shape) != (v, k // 256):
        raise RuntimeError("S must be [V, K/256]")
    return act.shape[0]


def fv5b_head_gemv_packed(wp, s, v: int, k: int, x, y=None, stream=None):
    """fv5b_head_gemv over the packed copy wp (i8_head_pack) of W [v,k]."""
    import torch
    m = _fv5b_packed_args(s, v, k, x, (torch.bfloat16, torch.int16, torch.uint16))
    if y is None:
        y = _new((m, v), torch.float32, x.device, stream)
    _check("fv5b_head_gemv_packed", lib().fv5b_head_gemv_packed(_ptr(wp), _ptr(s), v, k, _ptr(x), m, _ptr(y),
                                                                _stream(stream)))
    return y


def fv5b_head_gemv_packed_i8(wp, s, v: int, k: int, q, s_x, y=None, acc=None, stream=None):
    import torch
    m = _fv5b_packed_args(s, v, k, q, (torch.int8,))
    if y is None:
        y = _new((m, v), torch.float32, q.device, stream)
    _check("fv5b_head_gemv_packed_i8", lib().fv5b_head_gemv_packed_i8(_ptr(wp), _ptr(s), v, k, _ptr(q), _ptr(s_x),
                                                                      m, _ptr(y), _ptr(acc), _stream(stream)))
    return y


def fv5b_head_argmax_packed(wp, s, v: int, k: int, x, workspace=None, logits=None, stream=None):
    import torch
    m = _fv5b_packed_args(s, v, k, x, (torch.bfloat16, torch.int16, torch.uint16))
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, x.device, stream, returned=False)
    idx = _new(m, torch.int32, x.device, stream)
    val = _new(m, torch.float32, x.device, stream)
    _check("fv5b_head_argmax_packed", lib().fv5b_head_argmax_packed(_ptr(wp), _ptr(s), v, k, _ptr(x), m, _ptr(idx),
                                                                    _ptr(val), _ptr(logits), _ptr(workspace),
                                                                    _stream(stream)))
    return idx, val


def fv5b_head_argmax_packed_i8(wp, s, v: int, k: int, q, s_x, workspace=None, logits=None, stream=None):
    import torch
    m = _fv5b_packed_args(s, v, k, q, (torch.int8,))
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, q.device, stream, returned=False)
    idx = _new(m, torch.int32, q.device, stream)
    val = _new(m, torch.float32, q.device, stream)
    _check("fv5b_head_argmax_packed_i8", lib().fv5b_head_argmax_packed_i8(_ptr(wp), _ptr(s), v, k, _ptr(q),
                                                                          _ptr(s_x), m, _ptr(idx), _ptr(val),
                                                                          _ptr(logits), _ptr(workspace),
                                                                          _stream(stream)))
    return idx, val


def fv5b_head_argmax_embed(w, s, x, e, es, workspace=None, logits=None, f32=True, bf16=True, out=None,
                           out_bf16=None, stream=None):
    """Greedy argmax over the block-scaled head's logits of bf16 x, then the embedding rows of the chosen
    indices from the block-scaled table (e int8 [Ve,Ke], es fp32 [Ve,Ke/256]), in one call:
    (idx int32 [M], val fp32 [M], emb fp32 [M,Ke] or None, emb bf16 [M,Ke] or None)."""
    import torch
    v, k, m = _fv5b_args(w, s, x, (torch.bfloat16, torch.int16, torch.uint16))
    _need(e, "E", (torch.int8,), 2)
    _need(es, "ES", (torch.float32,), 2)
    ve, ke = e.shape
    if workspace is None:
        workspace = _new(i8_head_argmax_workspace_bytes(v, m), torch.uint8, x.device, stream, returned=False)
    idx = _new(m, torch.int32, x.device, stream)
    val = _new(m, torch.float32, x.device, stream)
    if out is None and f32:
        out = _new((m, ke), torch.float32, x.device, stream)
    if out_bf16 is None and bf16:
        out_bf16 = _new((m, ke), torch.bfloat16, x.device, stream)
    _check("fv5b_head_argmax_embed",
           lib().fv5b_head_argmax_embed(_ptr(w), _ptr(s), v, k, _ptr(x), m, _ptr(idx), _ptr(val), _ptr(logits),
                                        _ptr(workspace), _ptr(e), _ptr(es), ve, ke, _ptr(out), _ptr(out_bf16),
                                        _stream(stream)))
    return idx, val, out, out_bf16


def fv5b_embed(w, s, ids, f32=True, bf16=True, out=None, out_bf16=None, stream=None):
    """Embedding rows of int32 token ids [M]: (fp32 [M,K] or None, bf16 [M,K] or None); ids outside [0,V)
    give zeros.  Preallocated outputs may be passed as out / out_bf16."""
    import torch
    _need(w, "W", (torch.int8,), 2)
    _need(s, "S", (torch.float32,), 2)
    _need(ids, "ids", (torch.int32,), 1)
    v, k = w.shape
    m = ids.shape[0]
    if out is None and f32:
        out = _new((m, k), torch.float32, ids.device, stream)
    if out_bf16 is None and bf16:
        out_bf16 = _new((m, k), torch.bfloat16, ids.device, stream)
    _check("fv5b_embed", lib().fv5b_embed(_ptr(w), _ptr(s), v, k, _ptr(ids), m, _ptr(out), _ptr(out_bf16),
                                          _stream(stream)))
    return out, out_bf16


GEMV_KINDS = {"ternary_bf16": 0, "ternary_int8": 1, "fv5_bf16": 2, "fv5_int8": 3,
              "ternary_bf16_phased": 4, "ternary_int8_phased": 5, "fv5_bf16_phased": 6, "fv5_int8_phased": 7,
              "ternary_bf16_phased3": 8}


def tern_gemv_config(n: int, k: int, m: int, kind: str = "ternary_bf16"):
    """The one-pass launch configuration for this GEMV shape (host-side, no device needed), as a dict,
    or None when another kernel takes the shape."""
    out = (_i64 * 8)()
    rc = lib().tern_gemv_config(n, k, m, GEMV_KINDS[kind], out)
    if rc < 0:
        _check("tern_gemv_config", -rc)
    if rc == 0:
        return None
    keys = ("R", "waves", "U", "XC", "grid", "lds", "rounds", "MT")
    return dict(zip(keys, (int(v) for v in out)))


def tern_prefill_config(n: int, k: int, m: int):
    """The workgroup-shared-decode prefill launch for this shape (host-side, no device
    needed), as a dict, or None when another kernel takes the shape."""
    out = (_i64 * 6)()
    rc = lib().tern_prefill_config(n, k, m, out)
    if rc < 0:
        _check("tern_prefill_config", -rc)
    if rc == 0:
        return None
    keys = ("BM", "BN", "split", "grid_x", "grid_y", "grid_z")
    return dict(zip(keys, (int(v) for v in out)))


LAUNCH_PROBE_KINDS = {"empty": 0, "store": 1, "load": 2, "read": 3}


def tern_launch_probe(kind: str, grid: int, src=None, sink=None, stream=None):
    """Launch-floor / read-ceiling probe (measurement aid): enqueue one launch
    ("empty", "store": one float per workgroup, "load": one 16-byte load of
    src per thread first, "read": all of src read once by `grid` workgroups of
    256 threads).  src: a zero-filled device tensor (16-byte aligned); sink:
    at least `grid` floats (allocated when None)."""
    import torch
    if sink is None and kind != "empty":
        sink = _new(grid, torch.float32, "cuda", stream)
    nbytes = 0 if src is None else src.numel() * src.element_size()
    _check("tern_launch_probe", lib().tern_launch_probe(LAUNCH_PROBE_KINDS[kind], grid, _ptr(src), nbytes,
                                                         _ptr(sink), _stream(stream)))
    return sink


MFMA_PEAK_KINDS = {"int8": 0, "bf16": 1}


def tern_mfma_peak(kind: str, iters: int, grid: int, sink=None, stream=None):
    """Matrix-core throughput probe (measurement aid): enqueue one launch of
    `grid` workgroups running independent MFMA chains of `iters` steps
    ("int8": 16x16x64 i8, "bf16": 16x16x32 bf16).  Returns the operations the
    launch executes; time it with events on the same stream."""
    import torch
    k = MFMA_PEAK_KINDS[kind]
    ops = float(lib().tern_mfma_peak_ops(k, iters, grid))
    if ops < 0:
        _check("tern_mfma_peak", 2)
    if sink is None:
        sink = _new(int(lib().tern_mfma_peak_sink_bytes(grid)) // 4, torch.int32, "cuda", stream)
    _check("tern_mfma_peak", lib().tern_mfma_peak(k, iters, grid, _ptr(sink), _stream(stream)))
    return ops


# ---- attention over a paged int8 cache ----

# Per-call costs count here (a decode step's kernels take microseconds), so
# what torch is asked for per call is kept small: torch and the library's
# functions are looked up once, devices are compared by index, and the stream
# is taken as the number that the C ABI wants.
_torch = None
_TYPES = {}
_raw_stream = None


def _setup():
    global _torch, _TYPES, _raw_stream
    if _torch is None:
        import torch
        _TYPES = {torch.float32: 0, torch.bfloat16: 1}
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
        _torch = torch
    return _torch


def _vec(t, name, dtype, shape, device=None):
    """A contiguous device tensor of one dtype and shape (None: any size)."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA/HIP tensor")
    if t.shape == shape and t.dtype == dtype and t.get_device() == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise RuntimeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != len(shape) or any(w is not None and g != w for g, w in zip(t.shape, shape)):
        raise RuntimeError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise RuntimeError(f"{name} must be contiguous")
    if device is not None and t.get_device() != device:
        raise RuntimeError(f"{name} is on {t.device}, expected device {device}")


def _rows(t, name, dtype, device, heads, d, tokens):
    """A [T, heads, D] tensor whose rows may be strided and whose heads are contiguous: (T, heads, row
    stride).  dtype None: fp32 or bf16; heads or tokens None: any."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA/HIP tensor")
    if t.dtype != dtype if dtype is not None else t.dtype not in _TYPES:
        raise RuntimeError(f"{name} has dtype {t.dtype}, expected {dtype or 'float32 or bfloat16'}")
    shape = t.shape
    if len(shape) != 3:
        raise RuntimeError(f"{name} must be [T, heads, D]")
    n, h, dd = shape
    if dd != d or (heads is not None and h != heads) or (tokens is not None and n != tokens):
        raise RuntimeError(f"{name} has shape {tuple(shape)}, expected [{'T' if tokens is None else tokens}, "
                           f"{'heads' if heads is None else heads}, {d}]")
    if t.get_device() != device:
        raise RuntimeError(f"{name} is on {t.device}, expected device {device}")
    row, head, one = t.stride()
    if n and h and (one != 1 or (h > 1 and head != d)):
        raise RuntimeError(f"{name}: the heads of a row must be contiguous")
    return n, h, row if n > 1 else h * d


def _new(shape, dtype, device, stream, returned=True):
    """An output or a workspace for one call.  The memory comes from the stream that will write it: what
    the current stream has freed may still be in use there.  An output that is returned is kept from
    reuse until the current stream, the caller's, is done with it too."""
    torch = _torch or _setup()
    current = None if stream is None else torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(current)
    return t


def _call(name, device, stream, *args):
    """One library call on a device: made the current one where it is not, on its current stream or the
    one given (not one of another device, which the tensors need not be mapped on)."""
    if stream is None:
        handle = _raw_stream(device)
    elif stream.device_index == device:
        handle = stream.cuda_stream
    else:
        raise RuntimeError(f"stream is on device {stream.device_index}, expected {device}")
    f = getattr(_lib or lib(), name)
    if _torch.cuda.current_device() == device:
        rc = f(*args, handle)
    else:
        with _torch.cuda.device(device):
            rc = f(*args, handle)
    if rc:
        _check(name, rc)


def _addr(t):
    return None if t is None else t.data_ptr()


class QkTransform:
    """Norm gains (fp32 [D]), inverse frequencies (fp64 [D/2], radians per position) and rotation
    style of one layer's query and key heads; None leaves a part out."""

    def __init__(self, d: int, q_gain=None, k_gain=None, eps: float = 1e-6, inv_freq=None, interleaved: bool = False):
        torch = _setup()
        self.d, self.q_gain, self.k_gain, self.inv_freq = d, q_gain, k_gain, inv_freq
        self.device = None               # index; None: holds no tensor
        for t, name, dtype, n in ((q_gain, "q_gain", torch.float32, d), (k_gain, "k_gain", torch.float32, d),
                                  (inv_freq, "inv_freq", torch.float64, d // 2)):
            if t is not None:
                _vec(t, name, dtype, (n,), self.device)
                self.device = t.get_device()
        self.c = _QkTransform(_addr(q_gain), _addr(k_gain), _addr(inv_freq), eps, int(interleaved))
        self.ref = ctypes.byref(self.c)


class I8KvCache:
    """A paged int8 key/value cache: codes int8 [blocks, heads, 2, 64*D], scales fp32 [blocks, heads, 2]
    (one for each block of 64 tokens, head and side K, V).  Allocated here, or over tensors given."""

    def __init__(self, blocks: int = 0, heads: int = 0, d: int = 0, device="cuda", codes=None, scales=None):
        torch = _setup()
        if codes is None:
            codes = torch.zeros((blocks, heads, 2, KV_BLOCK * d), dtype=torch.int8, device=device)
            scales = torch.zeros((blocks, heads, 2), dtype=torch.float32, device=device)
        _vec(codes, "codes", torch.int8, (None, None, 2, None))
        blocks, heads, _, width = codes.shape
        if width not in (KV_BLOCK * 64, KV_BLOCK * 128):
            raise RuntimeError(f"codes hold {width} bytes a side, expected 64 * D with D 64 or 128")
        self.codes, self.scales, self.device = codes, scales, codes.get_device()
        _vec(scales, "scales", torch.float32, (blocks, heads, 2), self.device)
        self.blocks, self.heads, self.d = blocks, heads, width // KV_BLOCK
        self.c = _KvCache(codes.data_ptr(), scales.data_ptr(), blocks, heads, self.d)
        self.ref = ctypes.byref(self.c)


class I8KvBatch:
    """The sequences of a step: cu int32 [nseq+1] (rows cu[i]..cu[i+1]-1 are the newest tokens of
    sequence i), lens int32 [nseq] (lengths with them), table int32 [nseq, width] (their blocks).
    The kernels read all three, so they may be changed in place between calls."""

    def __init__(self, cu, lens, table):
        torch = _setup()
        _vec(cu, "cu", torch.int32, (None,))
        nseq = cu.shape[0] - 1
        if nseq < 0:
            raise RuntimeError("cu needs nseq + 1 entries")
        self.device = cu.get_device()
        _vec(lens, "lens", torch.int32, (nseq,), self.device)
        if not isinstance(table, torch.Tensor) or table.dtype != torch.int32 or table.get_device() != self.device:
            raise RuntimeError("table must be an int32 tensor on the device of cu")
        if table.dim() != 2 or table.shape[0] != nseq or (table.shape[1] > 1 and table.stride(1) != 1):
            raise RuntimeError(f"table has shape {tuple(table.shape)}, expected ({nseq}, width) with contiguous rows")
        self.cu, self.lens, self.table, self.nseq = cu, lens, table, nseq
        self.width = table.shape[1]
        stride = table.stride(0) if nseq > 1 else self.width
        self.c = _KvBatch(cu.data_ptr(), lens.data_ptr(), table.data_ptr(), nseq, self.width, stride)
        self.ref = ctypes.byref(self.c)


def qk_norm_rope(transform, q, k, pos=None, q_out=None, k_out=None, out_dtype=None, stream=None):
    """Norm and rotation of q [T, Hq, D] and k [T, Hk, D] (fp32 or bf16 rows, e.g. parts of one fused
    row; either may be None) at positions pos int32 [T]: (q, k) contiguous, out_dtype bf16 (default) or fp32."""
    x = q if q is not None else k
    if x is None:
        raise RuntimeError("qk_norm_rope: q or k is needed")
    device = transform.device
    if device is None:
        device = x.get_device() if isinstance(x, _torch.Tensor) else -1
    d = transform.d
    if out_dtype is None:
        out_dtype = q_out.dtype if q_out is not None else k_out.dtype if k_out is not None else _torch.bfloat16
    if out_dtype not in _TYPES:
        raise RuntimeError(f"out_dtype {out_dtype}, expected float32 or bfloat16")
    tokens = dtype = None
    hq = qs = hk = ks = 0
    if q is not None:
        tokens, hq, qs = _rows(q, "q", None, device, None, d, None)
        dtype = q.dtype
        if q_out is None:
            q_out = _new((tokens, hq, d), out_dtype, device, stream)
        else:
            _vec(q_out, "q_out", out_dtype, (tokens, hq, d), device)
    if k is not None:
        tokens, hk, ks = _rows(k, "k", dtype, device, None, d, tokens)
        dtype = k.dtype
        if k_out is None:
            k_out = _new((tokens, hk, d), out_dtype, device, stream)
        else:
            _vec(k_out, "k_out", out_dtype, (tokens, hk, d), device)
    if pos is not None:
        _vec(pos, "pos", _torch.int32, (tokens,), device)
    _call("qk_norm_rope", device, stream, transform.ref, tokens, d, _addr(q), hq, qs, _addr(k), hk, ks,
          _TYPES[dtype], _addr(pos), _addr(q_out) if q is not None else None,
          _addr(k_out) if k is not None else None, _TYPES[out_dtype])
    return (q_out if q is not None else None), (k_out if k is not None else None)


def _kv_device(cache, batch, transform=None):
    if batch.device != cache.device:
        raise RuntimeError(f"batch is on device {batch.device}, expected {cache.device}")
    if transform is not None and transform.device is not None and transform.device != cache.device:
        raise RuntimeError(f"transform is on device {transform.device}, expected {cache.device}")
    return cache.device


def i8_kv_append(cache, batch, transform, k, v, q=None, pos=None, q_out=None, stream=None):
    """Append k, v [T, heads, D] (fp32 or bf16 rows) to the cache, k normalised and rotated on the way;
    with q [T, Hq, D] also its norm and rotation -> q bf16 [T, Hq, D] (else None)."""
    device, d = _kv_device(cache, batch, transform), cache.d
    if transform.d != d:
        raise RuntimeError(f"transform is for D = {transform.d}, the cache for {d}")
    tokens, _, ks = _rows(k, "k", None, device, cache.heads, d, None)
    dtype = k.dtype
    vs = _rows(v, "v", dtype, device, cache.heads, d, tokens)[2]
    hq = qs = 0
    if q is not None:
        _, hq, qs = _rows(q, "q", dtype, device, None, d, tokens)
        if q_out is None:
            q_out = _new((tokens, hq, d), _torch.bfloat16, device, stream)
        else:
            _vec(q_out, "q_out", _torch.bfloat16, (tokens, hq, d), device)
    elif q_out is not None:
        raise RuntimeError("q_out without q")
    if pos is not None:
        _vec(pos, "pos", _torch.int32, (tokens,), device)
    _call("i8_kv_append", device, stream, cache.ref, batch.ref, transform.ref, tokens, _addr(q), hq, qs, k.data_ptr(),
          ks, v.data_ptr(), vs, _TYPES[dtype], _addr(pos), _addr(q_out))
    return q_out


def i8_kv_read(cache, batch, tokens: int, dtype=None, k_out=None, v_out=None, stream=None):
    """The batch's tokens (`tokens` rows) read back from the cache: (k, v) [T, heads, D], bf16 or fp32."""
    device = _kv_device(cache, batch)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else v_out.dtype if v_out is not None else _torch.bfloat16
    if dtype not in _TYPES:
        raise RuntimeError(f"dtype {dtype}, expected float32 or bfloat16")
    shape = (tokens, cache.heads, cache.d)
    if k_out is None:
        k_out = _new(shape, dtype, device, stream)
    else:
        _vec(k_out, "k_out", dtype, shape, device)
    if v_out is None:
        v_out = _new(shape, dtype, device, stream)
    else:
        _vec(v_out, "v_out", dtype, shape, device)
    _call("i8_kv_read", device, stream, cache.ref, batch.ref, tokens, k_out.data_ptr(), v_out.data_ptr(),
          _TYPES[dtype])
    return k_out, v_out


def i8_kv_attend_workspace_bytes(tokens: int, hq: int, heads: int, d: int, nseq: int, max_len: int,
                                 max_rows: int = 0) -> int:
    return int(lib().i8_kv_attend_workspace_bytes(tokens, hq, heads, d, nseq, max_len, max_rows))


def i8_kv_attend_workspace(cache, batch, tokens: int, hq: int, max_len=None, max_rows: int = 0):
    """A workspace for i8_kv_attend of `tokens` rows of hq heads (None where none is needed)."""
    nbytes = i8_kv_attend_workspace_bytes(tokens, hq, cache.heads, cache.d, batch.nseq,
                                          max_len or max(1, batch.width * KV_BLOCK), max_rows)
    if nbytes < 0:
        _check("i8_kv_attend_workspace_bytes", 2)
    return _torch.empty(nbytes, dtype=_torch.uint8, device=cache.device) if nbytes else None


def i8_kv_attend_config(tokens: int, hq: int, heads: int, d: int, nseq: int, width: int, window: int = 0,
                        max_len=None, max_rows: int = 0):
    """The launches that i8_kv_attend takes for `tokens` rows of hq heads (host-side, no device needed; width:
    of the table, max_len by default what that holds): a list of dicts, empty where there is nothing to do."""
    out = (_i64 * 12)()
    rc = lib().i8_kv_attend_config(tokens, hq, heads, d, nseq, width, window,
                                   max(1, width * KV_BLOCK) if max_len is None else max_len, max_rows, out)
    if rc < 0:
        _check("i8_kv_attend_config", -rc)
    keys = ("cols", "groups", "grid", "min_cols", "max_cols", "streams")
    return [dict(zip(keys, (int(v) for v in out[6 * i:6 * i + 6]))) for i in range(rc)]


def i8_kv_attend(cache, batch, q, scale=None, window: int = 0, max_len=None, max_rows: int = 0, out=None,
                 workspace=None, stream=None):
    """Attention of q bf16 [T, Hq, D] over the batch's cached tokens, causal, with a sliding window
    where window > 0 -> bf16 [T, Hq, D].  scale: D ** -0.5 by default.  Hints: max_len, the longest
    length that batch.lens will hold (default: what the table can hold), and max_rows, the most rows
    that a sequence will have (0: not known)."""
    device, d = _kv_device(cache, batch), cache.d
    tokens, hq, stride = _rows(q, "q", _torch.bfloat16, device, None, d, None)
    if max_len is None:
        max_len = batch.width * KV_BLOCK or 1
    if out is None:
        out = _new((tokens, hq, d), _torch.bfloat16, device, stream)
    else:
        _vec(out, "out", _torch.bfloat16, (tokens, hq, d), device)
    need = lib().i8_kv_attend_workspace_bytes(tokens, hq, cache.heads, d, batch.nseq, max_len, max_rows)
    if workspace is None:
        if need > 0:
            workspace = _new(need, _torch.uint8, device, stream, returned=False)
    elif workspace.get_device() != device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise RuntimeError(f"workspace must be a contiguous tensor of at least {need} bytes on device {device}")
    _call("i8_kv_attend", device, stream, cache.ref, batch.ref, tokens, q.data_ptr(), hq, stride,
          d ** -0.5 if scale is None else scale, window, max_len, max_rows, out.data_ptr(), _addr(workspace))
    return out
