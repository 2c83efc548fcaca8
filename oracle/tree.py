"""Trees of drafted tokens: CPU oracle in 64 bits, NumPy only, written from the
definitions in include/tern.h.  Test infrastructure."""
from __future__ import annotations

import numpy as np

from . import kv

ROWS = 512


def _sequences(cu, tokens):
    """(sequence, first row, rows) of those that the calls serve."""
    for i in range(len(cu) - 1):
        if cu[i + 1] < cu[i]:
            return
        if cu[i] >= 0 and cu[i + 1] <= tokens and cu[i + 1] > cu[i]:
            yield i, int(cu[i]), int(cu[i + 1] - cu[i])


def branch(parent, row):
    """Rows that `row` of a tree descends from, itself first."""
    out = []
    while row >= 0:
        out.append(row)
        p = int(parent[row])
        row = p if 0 <= p < row else -1
    return out


def mask(cu, lens, parent, words, before_mask, before_pos):
    """(mask uint64 [T][words], pos int32 [T]); rows of no sequence as before."""
    m, pos = np.array(before_mask, np.uint64), np.array(before_pos)
    for i, t0, n in _sequences(cu, len(parent)):
        p0 = max(int(lens[i]), 0) - n
        for j in range(n):
            m[t0 + j] = 0
            pos[t0 + j] = p0 + j
            if j < 64 * words:
                rows = branch(parent[t0:t0 + n], j)
                for r in rows:
                    m[t0 + j, r // 64] |= np.uint64(1 << (r % 64))
                pos[t0 + j] = p0 + len(rows) - 1
    return m, pos


def accept(cu, parent, token, target, width):
    nseq = len(cu) - 1
    path, count, following = np.full((nseq, width), -1, np.int32), np.zeros(nseq, np.int32), np.full(nseq, -1, np.int32)
    for i, t0, n in _sequences(cu, len(parent)):
        row, took = 0, []
        while True:
            took.append(row)
            if len(took) == width:
                break
            said = target[t0 + row]
            row = next((c for c in range(row + 1, min(n, ROWS)) if parent[t0 + c] == row and token[t0 + c] == said), -1)
            if row < 0:
                break
        path[i, :len(took)], count[i], following[i] = took, len(took), target[t0 + took[-1]]
    return path, count, following


def kept(path, rows):
    """Entries of a path up to the first that does not ascend or is no row of the tree."""
    out = []
    for r in path:
        if not (out[-1] if out else -1) < r < min(rows, ROWS):
            break
        out.append(int(r))
    return out


def keep(cache, cu, lens, table, tokens, paths):
    """Moves the paths' tokens in a kv.Cache -> lens_out.  Decisions in fp32, as the library takes them."""
    f = np.float32
    lens_out = np.maximum(lens, 0).astype(np.int32)

    def phys(i, position):
        b = position // kv.BLOCK
        return int(table[i, b]) if position >= 0 and b < table.shape[1] and 0 <= table[i, b] < cache.blocks else -1

    for i, t0, n in _sequences(cu, tokens):
        p0 = max(int(lens[i]), 0) - n
        path = kept(paths[i], n)
        lens_out[i] = max(p0 + len(path), 0)
        moved = [(p0 + k, p0 + r) for k, r in enumerate(path) if p0 + k >= 0]
        for block in sorted({to // kv.BLOCK for to, _ in moved}):
            mine = [(to, of) for to, of in moved if to // kv.BLOCK == block]
            dst = phys(i, block * kv.BLOCK)
            if dst < 0 or all(to == of for to, of in mine):
                continue
            for h in range(cache.heads):
                for side in (0, 1):
                    _keep(cache, [(to % kv.BLOCK, phys(i, of), of % kv.BLOCK) for to, of in mine], dst, h, side, f)
    return lens_out


def _keep(cache, mine, dst, h, side, f):
    codes = cache.tokens(dst, h, side)
    new = codes.copy()
    old = f(cache.scales[dst, h, side])
    far = {}
    with np.errstate(all="ignore"):
        for to, src, of in mine:
            if src >= 0 and src != dst:
                far[to] = cache.tokens(src, h, side)[of].astype(f) * f(cache.scales[src, h, side])
        strange = [f(cache.scales[src, h, side]) for _, src, _ in mine
                   if src >= 0 and src != dst and not np.isfinite(cache.scales[src, h, side])]
        top = max([np.abs(x).max() for x in far.values()], default=f(0)) if not strange else strange[0]
        if np.isinf(top):                                # code * scale past fp32
            strange = [top]
        scale, g, zero = old, 0, False
        if strange or top > 0:
            if old == 0:
                scale, zero = (top if strange else top / f(127)), True
            elif not np.isfinite(old) or strange:
                scale, zero = (old if not np.isfinite(old) else top), True
            else:
                while float(top) > np.ldexp(float(f(127) * old), g):     # 2^g alone may pass fp32
                    g += 1
                scale = f(np.ldexp(float(old), g))
        if zero:
            new[:] = 0
        elif g:
            new = np.rint(codes.astype(np.float64) / 2.0 ** g).astype(np.int8)
        source = new.copy()
        for to, src, of in mine:
            if src == dst:
                new[to] = source[of]
            elif src >= 0:
                new[to] = np.clip(np.rint(far[to] / scale), -127, 127) if scale > 0 and np.isfinite(scale) else 0
    cache.scales[dst, h, side] = scale
    cache.codes[dst, h, side][cache.place[side].ravel()] = new.ravel()


def attend(cache, cu, lens, table, q, scale, masks):
    """q [T, Hq, D], masks uint64 [T][words] -> (fp64 [T, Hq, D], NaN in rows of no sequence; a bound on what the
    library's narrower operands do to it, kv.attend's)."""
    out, bound = np.full(q.shape, np.nan), np.zeros(q.shape)
    group = q.shape[1] // cache.heads
    for i, t0, n in _sequences(cu, len(q)):
        p0 = int(lens[i]) - n
        k, v, there = cache.sequence(table[i], max(int(lens[i]), 0))
        at = np.arange(k.shape[0])
        for j in range(n):
            seen = there & (at < p0)
            for a in range(min(j + 1, 64 * masks.shape[1])):
                if 0 <= p0 + a < len(at) and int(masks[t0 + j, a // 64]) >> (a % 64) & 1:
                    seen[p0 + a] = there[p0 + a]
            for h in range(q.shape[1]):
                if not seen.any():
                    out[t0 + j, h] = 0
                    continue
                kk, vv, row = k[seen, h // group], v[seen, h // group], np.asarray(q[t0 + j, h], np.float64)
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ row * scale
                    w = np.exp(s - s.max())
                    out[t0 + j, h] = w @ vv / w.sum()
                    e = abs(scale) * np.abs(row).max() * 2.0 ** -15 * np.abs(kk).sum(1).max()
                    bound[t0 + j, h] = (2 * e + 2.0 ** -9) * np.abs(vv).max(0)
    return out, bound
