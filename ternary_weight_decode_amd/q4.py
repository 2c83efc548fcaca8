"""Linears with 4-bit weights and group scales: W[n,k] = t[n,k] * scale[n,k/group],
t in [-8, 7], groups of 32, 64 or 128 (``include/tern.h`` has the layout).

    packed = tw.q4_pack(t_int8, scale_fp16)                # once, at load time
    y = tw.q4_gemv(packed, N, K, group, x_bf16)            # x [M, K], M <= 16 -> fp32 [M, N]
    q, s_x = tw.tern_quantize_i8(x_bf16)
    y = tw.q4_gemv_i8(packed, N, K, group, q, s_x)         # int8 activations
"""
from __future__ import annotations

import functools

import ternary_weight_decode_amd as _tw

# A small product takes as long as its call: what the call needs is looked up once.
_torch = _tw._setup()
_lib = _tw.lib()
_bf16, _fp32, _int8 = _torch.bfloat16, _torch.float32, _torch.int8
_BITS16 = (_bf16, _torch.int16, _torch.uint16)


def q4_packed_bytes(n: int, k: int, group: int) -> int:
    return int(_lib.q4_packed_bytes(n, k, group))


@functools.lru_cache(maxsize=256)
def _bytes(n, k, group):
    nbytes = _lib.q4_packed_bytes(n, k, group)
    if nbytes < 0:
        _tw._check("q4_packed_bytes", 2)
    return nbytes


def q4_pack(t, scale, out=None, stream=None):
    """t int8 [N,K] in [-8,7], K % 128 == 0; scale fp16 bits [N,K/group] (int16/uint16/float16), group 32, 64
    or 128 -> 4-bit uint8 blob."""
    _tw._need(t, "t", (_int8,), 2)
    _tw._need(scale, "scale", (_torch.int16, _torch.uint16, _torch.float16), 2)
    n, k = t.shape
    groups = scale.shape[1]
    if scale.shape[0] != n or (groups == 0) != (k == 0) or (k and k % groups):
        raise RuntimeError(f"q4_pack: scale has shape {tuple(scale.shape)}, expected ({n}, {k} / group)")
    group = k // groups if k else 128
    nbytes = _bytes(n, k, group)
    device = t.get_device()
    if scale.get_device() != device:
        raise RuntimeError(f"scale is on {scale.device}, expected device {device}")
    if out is None:
        out = _tw._empty(_torch.uint8, device, stream, nbytes)
    else:
        _blob(out, "out", nbytes, device)
    _tw._launch(_lib.q4_pack, device, stream, t.data_ptr(), scale.data_ptr(), n, k, group, out.data_ptr())
    return out


def _blob(t, name, nbytes, device):
    if not isinstance(t, _torch.Tensor) or t.get_device() != device or t.nbytes < nbytes or not t.is_contiguous():
        raise RuntimeError(f"{name} must be a contiguous tensor of at least {nbytes} bytes on device {device}")


def _rows(x, name, dtypes, k):
    """Rows and device of activations [M, k]."""
    if not isinstance(x, _torch.Tensor) or not x.is_cuda:
        raise RuntimeError(f"{name} must be a CUDA/HIP tensor")
    if x.dtype not in dtypes:
        raise RuntimeError(f"{name} has dtype {x.dtype}, expected one of {dtypes}")
    if x.dim() != 2 or x.shape[1] != k or not x.is_contiguous():
        raise RuntimeError(f"{name} has shape {tuple(x.shape)}, expected contiguous [M, {k}]")
    return x.shape[0], x.get_device()


def q4_gemv(packed, n: int, k: int, group: int, x, y=None, stream=None):
    """y[m,n] = sum_g scale[n,g] sum_{k in g} t[n,k] x[m,k]; x bf16 [M,K], M <= 16 -> y fp32 [M,N]."""
    m, device = _rows(x, "x", _BITS16, k)
    _blob(packed, "packed", _bytes(n, k, group), device)
    if y is None:
        y = _tw._empty(_fp32, device, stream, m, n)
    else:
        _tw._vec(y, "y", _fp32, (m, n), device)
    _tw._launch(_lib.q4_gemv, device, stream, packed.data_ptr(), n, k, group, x.data_ptr(), m, y.data_ptr())
    return y


def q4_gemv_i8(packed, n: int, k: int, group: int, q, s_x, y=None, stream=None):
    """int8 activations: y = s_x[m] sum_g scale[n,g] acc[m,n,g], acc exact; q int8 [M,K], s_x fp32 [M]."""
    m, device = _rows(q, "q", (_int8,), k)
    _blob(packed, "packed", _bytes(n, k, group), device)
    _tw._vec(s_x, "s_x", _fp32, (m,), device)
    if y is None:
        y = _tw._empty(_fp32, device, stream, m, n)
    else:
        _tw._vec(y, "y", _fp32, (m, n), device)
    _tw._launch(_lib.q4_gemv_i8, device, stream, packed.data_ptr(), n, k, group, q.data_ptr(), s_x.data_ptr(), m,
                y.data_ptr())
    return y
