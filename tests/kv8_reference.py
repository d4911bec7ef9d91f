"""The 8-bit KV cache operators by their definitions, in numpy.

Writing and reading follow include/i2s.h step by step in binary32 (so a pool is
compared byte for byte); norms, rotations and attention are in 64 bits.
"""

import numpy as np

BLOCK = 16
F32 = np.float32


def slab_bytes(dim, page):
    return 2 * page * dim + (page // BLOCK * 8 + 31) // 32 * 32


class Pool:
    """A pool as numpy arrays: codes [pages, heads, 2, page, dim], scales [pages, heads, 2, page / 16]."""

    def __init__(self, raw, heads, dim, page):
        self.heads, self.dim, self.page = heads, dim, page
        self.raw = raw.reshape(-1, heads, slab_bytes(dim, page))
        n, plane = self.raw.shape[0], page * dim
        self.codes = self.raw[:, :, :2 * plane].view(np.int8).reshape(n, heads, 2, page, dim).copy()
        tail = self.raw[:, :, 2 * plane:2 * plane + page // 2]
        self.scales = np.ascontiguousarray(tail).view(F32).reshape(n, heads, 2, page // BLOCK).copy()

    def bytes(self):
        out = self.raw.copy()
        n, plane = out.shape[0], self.page * self.dim
        out[:, :, :2 * plane] = self.codes.reshape(n, self.heads, -1).view(np.uint8)
        out[:, :, 2 * plane:2 * plane + self.page // 2] = (
            np.ascontiguousarray(self.scales.reshape(n, self.heads, -1)).view(np.uint8))
        return out.reshape(-1)


def quantize(x, inv):
    """clamp(round(x * inv), -127, 127), the product in binary32, halves away from zero."""
    v = np.clip((x.astype(F32) * F32(inv)).astype(np.float64), -127, 127)
    return (np.sign(v) * np.floor(np.abs(v) + 0.5)).astype(np.int8)


def write(pool, table, kv_len, row_start, k, v):
    """k, v: rows x heads x dim float32 (already the values of their dtype)."""
    for s, length in enumerate(kv_len):
        n = row_start[s + 1] - row_start[s]
        start = max(0, length - n)
        skip = max(0, n - length)   # rows at negative positions
        for block in range(start // BLOCK, -(-length // BLOCK) if n else 0):
            lo, hi = max(start, block * BLOCK), min(length, (block + 1) * BLOCK)
            if lo >= hi:
                continue
            page = table[s][block * BLOCK // pool.page]
            if not 0 <= page < len(pool.raw):
                continue
            at, sub = block * BLOCK % pool.page, block * BLOCK % pool.page // BLOCK
            for which, x in enumerate((k, v)):
                for h in range(pool.heads):
                    rows = row_start[s] + skip + np.arange(lo, hi) - start
                    new, codes = x[rows, h], pool.codes[page, h, which]
                    held, old = lo - block * BLOCK, pool.scales[page, h, which, sub]
                    if not np.isfinite(new).all() or (held and np.isnan(old)):
                        scale, inv = F32(np.nan), None
                    else:
                        scale = max(F32(np.abs(new).max()), F32(1e-5)) / F32(127)
                        if held and old >= scale:
                            scale = old
                        inv = F32(1) / scale
                        if held and old != scale:
                            codes[at:at + held] = quantize(codes[at:at + held].astype(F32) * old, inv)
                    codes[at + held:at + held + hi - lo] = 0 if inv is None else quantize(new, inv)
                    pool.scales[page, h, which, sub] = scale


def cached(pool, table, s, length, which):
    """Values [length, heads, dim] in 64 bits (codes times scales, exact), NaN where a page is bad, and which are there."""
    pos = np.arange(length)
    page = np.asarray(table[s])[pos // pool.page]
    there = (page >= 0) & (page < len(pool.raw))
    page = np.where(there, page, 0)
    slot = pos % pool.page
    codes = pool.codes[page, :, which, slot].astype(np.float64)
    return codes * pool.scales[page, :, which, slot // BLOCK].astype(np.float64)[:, :, None], there


def attention(pool, table, kv_len, row_start, q, scale, causal, window):
    """(out, lse, sum p|v|, largest sum |q||k| * scale, tokens seen times the largest value that a block seen can hold)
    for each row and head, in 64 bits; rows of no sequence NaN."""
    rows, heads, dim = q.shape
    group = heads // pool.heads
    out, lse = np.full((rows, heads, dim), np.nan), np.full((rows, heads), np.nan)
    weight, size, reach = np.zeros((rows, heads, dim)), np.zeros((rows, heads)), np.zeros((rows, heads))
    for s, length in enumerate(kv_len):
        n = row_start[s + 1] - row_start[s]
        if n == 0:
            continue
        k, there = cached(pool, table, s, length, 0)
        v, _ = cached(pool, table, s, length, 1)
        pos = np.arange(length - n, length)[:, None]
        key = np.arange(length)
        page = np.where(there, np.asarray(table[s])[key // pool.page], 0)
        holds = 127.0 * pool.scales[page, :, 1, key % pool.page // BLOCK]
        seen = np.broadcast_to(there, (n, length)).copy()
        if causal:
            seen &= key <= pos
        if window:
            seen &= key > pos - window
        at = slice(row_start[s], row_start[s + 1])
        for h in range(heads):
            x = q[at, h].astype(np.float64)
            kh, vh = np.where(there[:, None], k[:, h // group], 0), np.where(there[:, None], v[:, h // group], 0)
            if length == 0:
                out[at, h], lse[at, h] = 0, -np.inf
                continue
            with np.errstate(invalid="ignore", divide="ignore"):
                score = np.where(seen, x @ kh.T * scale, -np.inf)
                top = score.max(1, keepdims=True)
                top = np.where(np.isneginf(top), 0, top)
                p = np.where(seen, np.exp(score - top), 0)
                total = p.sum(1, keepdims=True)
                lse[at, h] = np.where(total > 0, top + np.log(total), -np.inf)[:, 0]
                p = np.where(total > 0, p / total, 0)
            out[at, h] = p @ vh
            weight[at, h] = p @ np.abs(vh)
            reach[at, h] = seen.sum(1) * np.where(seen, holds[:, h // group], 0).max(1)
            size[at, h] = np.where(seen, np.abs(x) @ np.abs(kh).T * abs(scale), 0).max(1)
    return out, lse, weight, size, reach


def norm_rope(x, gamma, eps, positions, turns, interleaved):
    """rows x heads x dim in 64 bits; turns: Python integers, or empty for no rotation."""
    y = x.astype(np.float64)
    if gamma is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(F32(eps))) * gamma.astype(np.float64)
    half = len(turns)
    if half == 0:
        return y
    angle = np.array([[int(p) * int(t) % (1 << 64) / 2.0 ** 64 for t in turns] for p in positions]) * 2 * np.pi
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out = y.copy()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    return out
