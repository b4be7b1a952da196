"""Plain reference of the quantised key/value cache and the attention over it:
numpy in 64 bits, one request, head and row at a time.  Test infrastructure
only; shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

I4, I8 = 1, 3
QMAX = {I4: 7, I8: 127}


def quantise(x, elem):
    """Rows (..., D) of fp16 -> integer codes and one fp16 scale per row."""
    x = np.asarray(x, np.float16).astype(np.float64)
    x = np.where(np.isnan(x), 0.0, np.clip(x, -65504.0, 65504.0))
    q = QMAX[elem]
    s = (np.abs(x).max(-1) / q).astype(np.float16)
    s = np.where(s == 0, np.float16(1), s)
    c = np.clip(np.rint(x / s.astype(np.float64)[..., None]), -q - 1, q)
    return c.astype(np.int64), s


def pack(codes, elem):
    u = np.asarray(codes, np.int64) & (255 if elem == I8 else 15)
    if elem == I4:
        u = u[..., 0::2] + 16 * u[..., 1::2]
    return u.astype(np.uint8)


def unpack(rows, elem):
    b = np.asarray(rows, np.uint8).astype(np.int64)
    if elem == I8:
        return np.where(b > 127, b - 256, b)
    c = np.stack((b % 16, b // 16), -1).reshape(*b.shape[:-1], -1)
    return np.where(c > 7, c - 16, c)


class Cache:
    """Codes and scales by page, as the library lays them out."""

    def __init__(self, elem, D, Hkv, page_size, num_pages, table):
        row = D if elem == I8 else D // 2
        self.elem, self.D, self.Hkv, self.page_size = elem, D, Hkv, page_size
        self.table = np.asarray(table, np.int32)
        self.k = np.zeros((num_pages, Hkv, page_size, row), np.uint8)
        self.v = np.zeros_like(self.k)
        self.scale = np.ones((num_pages, Hkv, page_size, 2), np.float16)

    def at(self, b, p):
        return int(self.table[b, p // self.page_size]), p % self.page_size

    def write(self, b, p, k, v):
        """k, v: Hkv x D fp16 of position p."""
        g, s = self.at(b, p)
        for i, (pool, x) in enumerate(((self.k, k), (self.v, v))):
            c, sc = quantise(x, self.elem)
            pool[g, :, s] = pack(c, self.elem)
            self.scale[g, :, s, i] = sc

    def read(self, b, p):
        """K and V of position p, Hkv x D, in 64 bits."""
        g, s = self.at(b, p)
        return tuple(unpack(pool[g, :, s], self.elem) * self.scale[g, :, s, i].astype(np.float64)[:, None]
                     for i, pool in enumerate((self.k, self.v)))

    def commit(self, b, base, accepted):
        src = [self.at(b, base + a) for a in accepted]
        held = [(self.k[g, :, s].copy(), self.v[g, :, s].copy(), self.scale[g, :, s].copy()) for g, s in src]
        for i, (k, v, sc) in enumerate(held):
            g, s = self.at(b, base + i)
            self.k[g, :, s], self.v[g, :, s], self.scale[g, :, s] = k, v, sc


def attend(cache, b, q, ctx, seen, scale):
    """Rows q (n x Hq x D) of request b behind ctx positions; seen: n x n truth
    values among the call's own tokens.  Returns the outputs, sum w|v| / sum w
    (what rounding errors are measured by) and the largest sum |q||k| scale."""
    q = np.asarray(q, np.float64)
    n, Hq, D = q.shape
    G = Hq // cache.Hkv
    kv = [cache.read(b, p) for p in range(ctx + n)]
    out, mag, big = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n):
        ps = list(range(ctx)) + [ctx + j for j in range(n) if seen[i][j]]
        if not ps:
            continue
        for h in range(Hq):
            k = np.array([kv[p][0][h // G] for p in ps])
            v = np.array([kv[p][1][h // G] for p in ps])
            s = k @ q[i, h] * scale
            big[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
            w = np.exp(s - s.max())
            out[i, h] = w @ v / w.sum()
            mag[i, h] = w @ np.abs(v) / w.sum()
    return out, mag, big
