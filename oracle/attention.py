"""Rotary positions, the paged 8-bit key/value cache and attention over it (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Plain NumPy in fp64, token by token and row by row:

* ``rope``        -- pair i of a head turned by positions[axis[i]][t] * inv_freq[i];
* ``PagedCache``  -- pages of T tokens per head with one exponent e for the keys and one
  for the values: e is the smallest integer >= -126 with max|x| <= 127 * 2^e over the
  tokens a page has taken, codes are rint(x / 2^e) (ties to even), a page that already
  holds tokens keeps the larger of its exponent and the new one and its codes become
  rint(q * 2^(old - new)); a NaN or infinity poisons the page (its values read as NaN);
* ``attend``      -- softmax(scale * q k^T) v with causal and windowed views, rows that
  see nothing giving 0 and a log sum of -infinity.
"""
from __future__ import annotations

import math

import numpy as np

POISON = 1 << 20  # the exponent of a page that took a NaN or an infinity


def rope(x, positions, inv_freq, axis=None, interleaved=False) -> np.ndarray:
    """x [tokens][heads][dim], positions [axes][tokens], inv_freq [rot / 2] -> fp64."""
    x = np.asarray(x, dtype=np.float64)
    pos = np.asarray(positions, dtype=np.float64)
    inv = np.asarray(inv_freq, dtype=np.float64)
    half = inv.size
    y = x.copy()
    for i in range(half):
        ang = pos[0 if axis is None else int(axis[i])] * inv[i]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def page_exponent(amax: float) -> int:
    """Smallest integer e >= -126 with amax <= 127 * 2^e."""
    if not math.isfinite(amax):
        return POISON
    e = -126
    if amax > 0:
        e = max(math.frexp(amax)[1] - 9, -126)
    while amax > math.ldexp(127.0, e):
        e += 1
    return e


class PagedCache:
    def __init__(self, pages: int, page_tokens: int, heads: int, dim: int):
        self.pages, self.T, self.heads, self.dim = pages, page_tokens, heads, dim
        self.q = {s: np.zeros((pages, page_tokens, heads, dim)) for s in "kv"}
        self.e = {s: np.full((pages, heads), -126, dtype=np.int64) for s in "kv"}

    def write(self, table, start: int, k, v) -> None:
        """Tokens k, v [n][heads][dim] of one sequence at positions start, start + 1, ..."""
        n = len(k)
        p = start
        while p < start + n:
            slot = p % self.T
            m = min(self.T - slot, start + n - p)
            page = int(table[p // self.T])
            if 0 <= page < self.pages:
                for side, x in (("k", k), ("v", v)):
                    part = np.asarray(x[p - start:p - start + m], dtype=np.float64)
                    for h in range(self.heads):
                        self._put(side, page, slot, h, part[:, h])
            p += m

    def _put(self, side, page, slot, h, x) -> None:
        with np.errstate(invalid="ignore"):
            amax = float(np.max(np.abs(x))) if np.all(np.isfinite(x)) else math.inf
        e = page_exponent(amax)
        if slot:
            old = int(self.e[side][page, h])
            e = max(e, old)
            if e > old:
                kept = self.q[side][page, :slot, h]
                self.q[side][page, :slot, h] = 0.0 if e == POISON else np.rint(np.ldexp(kept, old - e))
        self.e[side][page, h] = e
        self.q[side][page, slot:slot + len(x), h] = 0.0 if e == POISON else np.rint(np.ldexp(x, -e))

    def read(self, table, start: int, n: int):
        """(k, v) of n positions, fp64 [n][heads][dim]; NaN for poisoned pages and for page
        numbers outside the pool."""
        out = {s: np.full((n, self.heads, self.dim), np.nan) for s in "kv"}
        for i in range(n):
            page, slot = int(table[(start + i) // self.T]), (start + i) % self.T
            if not 0 <= page < self.pages:
                continue
            for s in "kv":
                for h in range(self.heads):
                    e = int(self.e[s][page, h])
                    if e != POISON:
                        out[s][i, h] = np.ldexp(self.q[s][page, slot, h], e)
        return out["k"], out["v"]


def attend(q, k, v, scale: float, causal: bool = True, window: int = 0):
    """q [n][q_heads][dim], k, v [kv][heads][dim] (fp64): (out, lse [n][q_heads], and the
    bound inputs of a tolerance: sum p |v| and max scale * sum |q||k| per row)."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, hq, dim = q.shape
    kv = k.shape[0]
    G = hq // k.shape[1] if k.shape[1] else 1
    out, mass = np.zeros((n, hq, dim)), np.zeros((n, hq, dim))
    lse, size = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for i in range(n):
        pos = kv - n + i
        hi = min(pos + 1, kv) if causal else kv
        lo = max(0, pos - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(hq):
            K, V = k[lo:hi, h // G], v[lo:hi, h // G]
            s = scale * (K @ q[i, h])
            m = np.max(s)
            w = np.exp(s - m)
            l = np.sum(w)
            out[i, h] = (w / l) @ V
            mass[i, h] = (w / l) @ np.abs(V)
            lse[i, h] = m + math.log(l) if not math.isnan(l) else math.nan
            size[i, h] = abs(scale) * np.max(np.abs(K) @ np.abs(q[i, h]))
    return out, lse, mass, size
