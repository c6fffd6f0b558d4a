"""Oracle: the 8-bit key/value cache, block attention and eviction (test
infrastructure), numpy float64 from the definitions in include/dllm_commit.h.
"""
import math

import numpy as np

PAGE = 32


def scale_of(x):
    """The page's scale: the smallest power of two s in [2^-100, 2^119] with
    |x| <= 448 s over its finite elements."""
    a = np.abs(x[np.isfinite(x)])
    amax = float(a.max()) if a.size else 0.0
    e = -100
    while e < 119 and amax > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


def e4m3_values():
    """The finite non-negative e4m3 values, ascending."""
    v = [m / 8.0 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:-1])          # the last code is NaN


_GRID = e4m3_values()


def code(x, s):
    """x / s rounded to the nearest e4m3 value (ties to the even code), times s."""
    v = np.where(np.isnan(x), 0.0, x) / s
    a = np.minimum(np.abs(v), 448.0)
    i = np.searchsorted(_GRID, a, side="right") - 1
    j = np.minimum(i + 1, len(_GRID) - 1)
    lo, hi = _GRID[i], _GRID[j]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
    q = np.where(up, hi, lo)
    return np.copysign(q, v) * s


class Cache:
    """The values of a pool: (pages, heads, 32, D) for keys and for values."""

    def __init__(self, pages, heads, dim):
        self.x = np.zeros((2, pages, heads, PAGE, dim))
        self.s = np.ones((2, pages, heads))

    def write(self, k, v, table, start, lens=None):
        B, L = k.shape[:2]
        for b in range(B):
            n = L if lens is None else min(int(lens[b]), L)
            s0 = int(start[b])
            if s0 < 0 or n <= 0:
                continue
            for p in range(s0 // PAGE, (s0 + n - 1) // PAGE + 1):
                if p >= table.shape[1] or not 0 <= table[b, p] < self.x.shape[1]:
                    continue
                page = table[b, p]
                lo, hi = max(0, s0 - p * PAGE), min(PAGE, s0 + n - p * PAGE)
                for i, src in enumerate((k, v)):
                    new = src[b, p * PAGE + lo - s0:p * PAGE + hi - s0]
                    for h in range(src.shape[2]):
                        s = scale_of(new[:, h])
                        if lo > 0:
                            s = max(s, self.s[i, page, h])
                            self.x[i, page, h, :lo] = code(self.x[i, page, h, :lo], s)
                        self.x[i, page, h, lo:hi] = code(new[:, h], s)
                        self.s[i, page, h] = s

    def read(self, table, lens):
        B, P = table.shape
        H, _, D = self.x.shape[2:]
        out = np.zeros((2, B, P * PAGE, H, D))
        for b in range(B):
            n = min(max(int(lens[b]), 0), P * PAGE)
            for t in range(n):
                page = table[b, t // PAGE]
                if 0 <= page < self.x.shape[1]:
                    out[:, b, t] = self.x[:, page, :, t % PAGE]
        return out[0], out[1]

    def gather(self, table, kept, counts, new_table):
        k, v = self.read(table, np.full(table.shape[0], table.shape[1] * PAGE))
        for b in range(table.shape[0]):
            n = min(max(int(counts[b]), 0), new_table.shape[1] * PAGE)
            for p in range((n + PAGE - 1) // PAGE):
                page = new_table[b, p]
                if not 0 <= page < self.x.shape[1]:
                    continue
                for i, src in enumerate((k, v)):
                    new = np.zeros((PAGE,) + src.shape[2:])
                    for j in range(PAGE):
                        if p * PAGE + j < n and 0 <= kept[b, p * PAGE + j] < src.shape[1]:
                            new[j] = src[b, kept[b, p * PAGE + j]]
                    for h in range(src.shape[2]):
                        s = scale_of(new[:, h])
                        self.x[i, page, h] = code(new[:, h], s)
                        self.s[i, page, h] = s


def live_tokens(table, n, pages):
    """Token positions of one sequence that are there: below n, on a real page."""
    T = table.shape[0] * PAGE
    t = np.arange(T)
    return (t < min(max(int(n), 0), T)) & (table[t // PAGE] >= 0) & (table[t // PAGE] < pages)


def block_attention(q, k, v, table, kv_lens, pages, q_start=None, q_lens=None, block_len=0,
                    scale=None):
    """q (B, L, Hq, D), k and v (B, T, H, D) the cached values.  Returns out, lse
    (B, Hq, L), weights (B, T), and per output the bounds a rounding analysis
    needs: sum p |v| and max over tokens of scale sum |q k|."""
    B, L, Hq, D = q.shape
    H = k.shape[2]
    G = Hq // H
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    T = k.shape[1]
    out, mass = np.zeros((B, L, Hq, D)), np.zeros((B, L, Hq, D))
    lse, mag = np.full((B, Hq, L), -np.inf), np.zeros((B, Hq, L))
    weights = np.zeros((B, T))
    for b in range(B):
        there = live_tokens(table[b], kv_lens[b], pages)
        for l in range(L if q_lens is None else min(int(q_lens[b]), L)):
            ok = there.copy()
            if block_len > 0:
                pos = (0 if q_start is None else max(int(q_start[b]), 0)) + l
                ok &= np.arange(T) // block_len <= pos // block_len
            t = np.flatnonzero(ok)
            if t.size == 0:
                continue
            for h in range(Hq):
                kk, vv = k[b, t, h // G], v[b, t, h // G]
                s = scale * (kk @ q[b, l, h])
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                p = e / z
                out[b, l, h] = p @ vv
                mass[b, l, h] = p @ np.abs(vv)
                lse[b, h, l] = m + np.log(z)
                mag[b, h, l] = scale * (np.abs(kk) @ np.abs(q[b, l, h])).max()
                weights[b, t] += p
    return out, lse, weights, mass, mag


def evict_select(weights, lens, budget, sink=0, recent=0):
    B, T = weights.shape
    kept = np.full((B, budget), -1, dtype=np.int32)
    new_lens = np.zeros(B, dtype=np.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), T)
        w = np.where(np.isnan(weights[b]), -np.inf, weights[b]) + 0.0
        if n <= budget:
            keep = list(range(n))
        else:
            order = sorted(range(n), key=lambda t: (not (t < sink or t >= n - recent),
                                                    -w[t] if sink <= t < n - recent else 0, t))
            keep = sorted(order[:budget])
        kept[b, :len(keep)] = keep
        new_lens[b] = len(keep)
    return kept, new_lens
