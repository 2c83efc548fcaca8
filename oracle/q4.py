"""4-bit weights with group scales: CPU oracle in 64 bits, NumPy only, written
from the definition in include/tern.h.  Test infrastructure."""
from __future__ import annotations

import numpy as np


def _npad(n: int) -> int:
    return (n + 15) // 16 * 16


def packed_bytes(n: int, k: int, group: int) -> int:
    if n < 0 or k < 0 or k % 128 or group not in (32, 64, 128):
        return -1
    return _npad(n) * k // 2 + 2 * _npad(n) * (k // group)


def pack(t, scale) -> np.ndarray:
    """t int [N][K] (clamped to [-8, 7]), scale fp16 [N][K/group] -> blob bytes."""
    n, k = t.shape
    group = k // scale.shape[1]
    nb, per = k // 128, 128 // group
    words = np.zeros(_npad(n) * k // 8, np.uint32)
    scales = np.zeros(_npad(n) * (k // group), np.uint16)
    bits = np.asarray(scale, np.float16).view(np.uint16)
    for row in range(n):
        rt, r = divmod(row, 16)
        for kk in range(k):
            b, rest = divmod(kk, 128)
            c, rest = divmod(rest, 32)
            g, i = divmod(rest, 8)
            v = min(7, max(-8, int(t[row, kk]))) % 16
            words[(rt * nb + b) * 256 + (g * 16 + r) * 4 + c] |= np.uint32(v << (16 * (i & 1) + 4 * (i >> 1)))
        for gr in range(k // group):
            b, j = divmod(gr, per)
            kt, bq = divmod(b, 4)
            nbq = min(4, nb - 4 * kt)
            scales[((rt * nb + 4 * kt) * 16 + r * nbq + bq) * per + j] = bits[row, gr]
    return np.concatenate([words.view(np.uint8), scales.view(np.uint8)])


def dense(t, scale) -> np.ndarray:
    group = t.shape[1] // scale.shape[1]
    return np.clip(t, -8, 7).astype(np.float64) * np.repeat(np.asarray(scale, np.float64), group, 1)


def gemv(t, scale, x):
    """x [M][K] -> (y fp64 [M][N], a bound on the error of q4_gemv).

    The bound: a group's products (exact, but for what x loses in fp16: 2^-39 of
    the largest of its 512 neighbours) are summed in fp32 in any order, 128 of
    them with an error of at most one step, 2^-23, of the sum of their sizes
    each; the scale's product and the sum over the groups add one rounding
    each, and the waves' partial sums 16."""
    w = dense(t, scale)
    x = np.asarray(x, np.float64)
    k = w.shape[1]
    y = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    bound = (128 * 2.0 ** -23 + (scale.shape[1] + 20) * 2.0 ** -24) * size
    for lo in range(0, k, 512):
        top = np.abs(x[:, lo:lo + 512]).max(1)
        bound += 2.0 ** -39 * top[:, None] * np.abs(w[:, lo:lo + 512]).sum(1)[None]
    return y, bound


def gemv_i8(t, scale, q, s_x):
    """q int8 [M][K], s_x fp32 [M] -> (y fp64 [M][N], bound): the groups' sums are exact, then one rounding for
    each product and sum."""
    n, k = t.shape
    groups = scale.shape[1]
    group = k // groups
    tt = np.clip(t, -8, 7).astype(np.int64).reshape(n, groups, group)
    acc = np.einsum("ngi,mgi->mng", tt, np.asarray(q, np.int64).reshape(len(q), groups, group))
    part = acc * np.asarray(scale, np.float64)[None]
    s = np.asarray(s_x, np.float64)[:, None]
    return part.sum(-1) * s, (groups + 20) * 2.0 ** -24 * np.abs(part).sum(-1) * np.abs(s)
