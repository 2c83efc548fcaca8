"""Independent 64-bit oracle of the attention side of a decode step: query/key
norm with rotation, the paged int8 cache's append and read, and attention
over it.  NumPy only; the definitions are those of include/tern.h."""
from __future__ import annotations

import numpy as np

BLOCK = 64


def bf16(x):
    """float -> the nearest bf16 value (ties to even), as float32."""
    x = np.ascontiguousarray(x, np.float32)
    u = x.view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)).view(np.float32)
    return np.where(np.isnan(x), x, r).astype(np.float32)


def transform(x, gain, eps, inv_freq, interleaved, pos):
    """x [T, heads, D] -> fp64; gain or inv_freq None leaves that part out."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    if inv_freq is None:
        return x
    a = np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(a), np.sin(a)
    y = np.empty_like(x)
    i1 = np.arange(0, d, 2) if interleaved else np.arange(d // 2)
    i2 = i1 + 1 if interleaved else i1 + d // 2
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def place(side, d):
    """Byte of every (token, dim) of a block: [64, D]."""
    out = np.empty((BLOCK, d), np.int64)
    for token in range(BLOCK):
        for dim in range(d):
            if side == 0:
                t, r = divmod(token, 16)
                s, rest = divmod(dim, 64)
                g, b = divmod(rest, 16)
                out[token, dim] = (((t * (d // 64) + s) * 4 + g) * 16 + r) * 16 + b
            else:
                t, rest = divmod(token, 16)
                g, i = divmod(rest, 4)
                u, r = divmod(dim, 16)
                out[token, dim] = ((u * 4 + g) * 16 + r) * 16 + 4 * t + i
    return out


class Cache:
    """A paged cache in host memory: codes int8 [blocks, heads, 2, 64*D], scales fp32 [blocks, heads, 2]."""

    def __init__(self, codes, scales):
        self.codes, self.scales = np.array(codes), np.array(scales)
        self.blocks, self.heads = codes.shape[:2]
        self.d = codes.shape[3] // BLOCK
        self.place = [place(0, self.d), place(1, self.d)]

    def tokens(self, phys, head, side):
        """Codes [64, D] of a block (a copy)."""
        return self.codes[phys, head, side][self.place[side]]

    def append(self, cu, lens, table, k, v):
        """k, v [T, heads, D]: the values as the cache receives them (k transformed).  Decisions in
        the precision of k and v: fp32 arrays give the library's bytes."""
        for i in range(len(lens)):
            n, p0 = cu[i + 1] - cu[i], lens[i] - (cu[i + 1] - cu[i])
            for b in range(p0 // BLOCK, (p0 + n - 1) // BLOCK + 1) if n > 0 else ():
                lo, hi = max(p0, b * BLOCK), min(p0 + n, (b + 1) * BLOCK)
                if b < 0 or b >= table.shape[1] or not 0 <= table[i, b] < self.blocks:
                    continue
                for h in range(self.heads):
                    for side, x in enumerate((k, v)):
                        rows = x[cu[i] + lo - p0:cu[i] + hi - p0, h]
                        self._join(table[i, b], h, side, lo - b * BLOCK, rows)

    def _join(self, phys, h, side, o, rows):
        f = rows.dtype.type
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            top = np.abs(rows).max()                     # NaN wins
            old = f(self.scales[phys, h, side])
            codes = self.tokens(phys, h, side)
            if o == 0 or old == 0:
                scale = top / f(127) if np.isfinite(top) else top
            elif not np.isfinite(old) or not np.isfinite(top):
                scale = top if np.isfinite(old) else old
                codes[:o] = 0
            else:
                g = 0
                while top > f(127) * old * f(2.0 ** g):
                    g += 1
                scale = old * f(2.0 ** g)
                codes[:o] = np.rint(codes[:o].astype(np.float64) / 2.0 ** g)
            if scale > 0 and np.isfinite(scale):
                codes[o:o + len(rows)] = np.clip(np.rint(rows / scale), -127, 127)
            else:
                codes[o:o + len(rows)] = 0
        self.scales[phys, h, side] = scale
        self.codes[phys, h, side][self.place[side].ravel()] = codes.ravel()

    def read(self, cu, lens, table, tokens):
        """K and V fp64 [tokens, heads, D] of the batch's rows (zeros where there is no cached token)."""
        out = np.zeros((2, tokens, self.heads, self.d))
        for i in range(len(lens)):
            n, p0 = cu[i + 1] - cu[i], lens[i] - (cu[i + 1] - cu[i])
            for j in range(n):
                p = p0 + j
                b = p // BLOCK
                if p < 0 or b >= table.shape[1] or not 0 <= table[i, b] < self.blocks:
                    continue
                for h in range(self.heads):
                    for side in (0, 1):
                        row = self.codes[table[i, b], h, side][self.place[side][p % BLOCK]]
                        out[side, cu[i] + j, h] = row * np.float64(self.scales[table[i, b], h, side])
        return out

    def sequence(self, row, length):
        """K, V fp64 [length, heads, D] of one sequence and which of its positions are cached."""
        k = np.zeros((length, self.heads, self.d))
        v = np.zeros_like(k)
        there = np.zeros(length, bool)
        for b in range(min(-(-length // BLOCK), len(row))):
            if not 0 <= row[b] < self.blocks:
                continue
            lo, hi = b * BLOCK, min(length, (b + 1) * BLOCK)
            there[lo:hi] = True
            for h in range(self.heads):
                for side, x in enumerate((k, v)):
                    x[lo:hi, h] = (self.tokens(row[b], h, side)[:hi - lo]
                                   * np.float64(self.scales[row[b], h, side]))
        return k, v, there


def attend(cache, cu, lens, table, q, scale, window=0):
    """q [T, Hq, D] -> fp64 [T, Hq, D] (NaN rows of no sequence), and a bound on the part of an output's error
    that the library's narrower operands cause, [T, Hq, D].

    The bound: q in 15 bits of its largest value moves a score by at most
    scale * max|q| * 2^-15 * sum|k|, a score's error e moves a weighted mean
    by at most 2 e max|v|, and weights held to 2^-15 of their block's largest
    (64 tokens) or to 2^-12 of themselves, with V to 2^-12 of itself, by at
    most 64 * 2^-15 max|v| = 2^-9 max|v|."""
    out = np.full(q.shape, np.nan)
    bound = np.zeros(q.shape)
    group = q.shape[1] // cache.heads
    for i in range(len(lens)):
        n, p0 = cu[i + 1] - cu[i], lens[i] - (cu[i + 1] - cu[i])
        if n == 0:
            continue
        k, v, there = cache.sequence(table[i], max(lens[i], 0))
        for j in range(n):
            p = p0 + j
            at = np.arange(k.shape[0])
            seen = there & (at <= p)
            if window:
                seen &= at > p - window
            for h in range(q.shape[1]):
                row = np.asarray(q[cu[i] + j, h], np.float64)
                if not seen.any():
                    out[cu[i] + j, h] = 0
                    continue
                kk, vv = k[seen, h // group], v[seen, h // group]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ row * scale
                    w = np.exp(s - s.max())
                    out[cu[i] + j, h] = w @ vv / w.sum()
                    e = abs(scale) * np.abs(row).max() * 2.0 ** -15 * np.abs(kk).sum(1).max()
                    bound[cu[i] + j, h] = (2 * e + 2.0 ** -9) * np.abs(vv).max(0)
    return out, bound
