"""Linears with 4-bit weights and group scales: W[n,k] = t[n,k] * scale[n,k/group],
t in [-8, 7], groups of 32, 64 or 128 (``include/tern.h`` has the layout).

    packed = tw.q4_pack(t_int8, scale_fp16)                # once, at load time
    y = tw.q4_gemv(packed, N, K, group, x_bf16)            # x [M, K], M <= 16 -> fp32 [M, N]
    q, s_x = tw.tern_quantize_i8(x_bf16)
    y = tw.q4_gemv_i8(packed, N, K, group, q, s_x)         # int8 activations
"""
from __future__ import annotations

import ternary_weight_decode_amd as _tw

_torch = _tw._setup()
_ACTIVATIONS = (_torch.bfloat16, _torch.int16, _torch.uint16)


def q4_packed_bytes(n: int, k: int, group: int) -> int:
    return int(_tw.lib().q4_packed_bytes(n, k, group))


def q4_pack(t, scale, out=None, stream=None):
    """t int8 [N,K] in [-8,7], K % 128 == 0; scale fp16 bits [N,K/group] (int16/uint16/float16), group 32, 64
    or 128 -> 4-bit uint8 blob."""
    _tw._need(t, "t", (_torch.int8,), 2)
    _tw._need(scale, "scale", (_torch.int16, _torch.uint16, _torch.float16), 2)
    n, k = t.shape
    groups = scale.shape[1]
    if scale.shape[0] != n or (groups == 0) != (k == 0) or (k and k % groups):
        raise RuntimeError(f"q4_pack: scale has shape {tuple(scale.shape)}, expected ({n}, {k} / group)")
    group = k // groups if k else 128
    nbytes = q4_packed_bytes(n, k, group)
    if nbytes < 0:
        _tw._check("q4_pack", 2)
    device = t.get_device()
    if scale.get_device() != device:
        raise RuntimeError(f"scale is on {scale.device}, expected device {device}")
    if out is None:
        out = _tw._new(nbytes, _torch.uint8, device, stream)
    else:
        _blob(out, "out", nbytes, device)
    _tw._call("q4_pack", device, stream, t.data_ptr(), scale.data_ptr(), n, k, group, out.data_ptr())
    return out


def _blob(t, name, nbytes, device):
    if not isinstance(t, _torch.Tensor) or t.get_device() != device or not t.is_contiguous() or \
            t.numel() * t.element_size() < nbytes:
        raise RuntimeError(f"{name} must be a contiguous tensor of at least {nbytes} bytes on device {device}")


def _linear(name, packed, n, k, group, x, dtypes, y, stream):
    """(M, device, y) of a product with activations x [M, K]."""
    if not isinstance(x, _torch.Tensor) or not x.is_cuda:
        raise RuntimeError("the activations must be a CUDA/HIP tensor")
    shape = x.shape
    if x.dtype not in dtypes:
        raise RuntimeError(f"the activations have dtype {x.dtype}, expected one of {dtypes}")
    if len(shape) != 2 or shape[1] != k or not x.is_contiguous():
        raise RuntimeError(f"the activations have shape {tuple(shape)}, expected contiguous [M, {k}]")
    device, m = x.get_device(), shape[0]
    nbytes = _tw.lib().q4_packed_bytes(n, k, group)
    if nbytes < 0:
        _tw._check(name, 2)
    _blob(packed, "packed", nbytes, device)
    if y is None:
        y = _tw._new((m, n), _torch.float32, device, stream)
    else:
        _tw._vec(y, "y", _torch.float32, (m, n), device)
    return m, device, y


def q4_gemv(packed, n: int, k: int, group: int, x, y=None, stream=None):
    """y[m,n] = sum_g scale[n,g] sum_{k in g} t[n,k] x[m,k]; x bf16 [M,K], M <= 16 -> y fp32 [M,N]."""
    m, device, y = _linear("q4_gemv", packed, n, k, group, x, _ACTIVATIONS, y, stream)
    _tw._call("q4_gemv", device, stream, packed.data_ptr(), n, k, group, x.data_ptr(), m, y.data_ptr())
    return y


def q4_gemv_i8(packed, n: int, k: int, group: int, q, s_x, y=None, stream=None):
    """int8 activations: y = s_x[m] sum_g scale[n,g] acc[m,n,g], acc exact; q int8 [M,K], s_x fp32 [M]."""
    m, device, y = _linear("q4_gemv_i8", packed, n, k, group, q, (_torch.int8,), y, stream)
    _tw._vec(s_x, "s_x", _torch.float32, (m,), device)
    _tw._call("q4_gemv_i8", device, stream, packed.data_ptr(), n, k, group, q.data_ptr(), s_x.data_ptr(), m,
              y.data_ptr())
    return y
