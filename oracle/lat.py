"""Plain reference of the page pool, of norm and rotation, and of the attention over
latent and over expanded rows: Python and numpy in 64 bits.  Test infrastructure only;
shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np


class Pool:
    """Pages held by requests and a stack of free ones, one page at a time."""

    def __init__(self, page_size, num_pages, B, max_pages):
        self.page_size, self.max_pages = page_size, max_pages
        self.held = [[] for _ in range(B)]
        self.free = list(range(num_pages - 1, -1, -1))

    def reserve(self, lengths):
        """Whether every request got what it wanted."""
        want = [-(-n // self.page_size) for n in lengths]
        for b, w in enumerate(want):
            back, self.held[b] = self.held[b][w:], self.held[b][:w]
            self.free += back
        short = False
        for b, w in enumerate(want):
            more = w - len(self.held[b])
            if more > 0 and (short or more > len(self.free)):
                short = True
                continue
            for _ in range(more):
                self.held[b].append(self.free.pop())
        return not short

    def table(self):
        t = np.full((len(self.held), self.max_pages), -1, np.int32)
        for b, pages in enumerate(self.held):
            t[b, :len(pages)] = pages
        return t

    def slot(self, b, p):
        return self.held[b][p // self.page_size] * self.page_size + p % self.page_size


def norm(x, w, eps):
    """Rows (..., D); w None: as they are."""
    x = np.asarray(x).astype(np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w).astype(np.float64)


def rotate(x, p, freq, pairs):
    """x (T x ... x D) with its first 2 len(freq) values turned by positions p (T) times freq (radians)."""
    x = np.array(x, np.float64)
    R = 2 * len(freq)
    if R == 0:
        return x
    angle = np.asarray(p, np.float64).reshape(-1, *[1] * (x.ndim - 1)) * np.asarray(freq, np.float64)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if pairs else (slice(0, R // 2), slice(R // 2, R))
    u, v = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * np.cos(angle) - v * np.sin(angle)
    x[..., b] = v * np.cos(angle) + u * np.sin(angle)
    return x


def attend(q, k, v, seen, scale):
    """Rows q (n x W) over keys k (L x W) and values v (L x D) where seen (n x L).

    Returns the outputs, the weighted mean of |v| and the largest sum of |q||k| scale a row."""
    q, k, v = (np.asarray(x).astype(np.float64) for x in (q, k, v))
    seen = np.asarray(seen, bool)
    s = np.where(seen, q @ np.where(seen.any(0)[:, None], k, 0).T * scale, -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    w = np.exp(s - np.where(np.isfinite(top), top, 0))
    total = w.sum(-1, keepdims=True)
    w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    vz = np.where(seen.any(0)[:, None], v, 0)
    big = np.abs(q) @ np.abs(np.where(seen.any(0)[:, None], k, 0)).T * abs(scale)
    return w @ vz, w @ np.abs(vz), np.where(seen, big, 0).max(-1, initial=0)
