"""Float64 oracle of rotary positions and the paged key/value cache.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see attn_f64).  Everything is the
definition written out: rotations as complex products, attention row by row
over the keys gathered through the page table, page operations on Python lists.
"""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ rotary positions
def rope_frequencies(axes, base=10000.0, factor=1.0, ramp=None):
    """Angle per position of each pair, and the axis of each pair."""
    freq, axis = [], []
    for a, d in enumerate(axes):
        for j in range(d // 2):
            f = base ** (-2.0 * j / d)
            if ramp is None:
                f = f / factor
            else:
                low, high, length = ramp
                w = (length * f / (2.0 * math.pi) - low) / (high - low)
                w = min(1.0, max(0.0, w))
                f = f * w + f * (1.0 - w) / factor
            freq.append(f)
            axis.append(a)
    return np.array(freq), np.array(axis)


def rope_pairs(n_pairs, interleaved):
    """Columns of the first and second element of each pair."""
    i = np.arange(n_pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + n_pairs)


def rope(x, positions, axes, base=10000.0, interleaved=False, factor=1.0, ramp=None, magnitude=1.0, sign=1):
    """x [T, H, d], positions [n_axes, T].  sign = -1: the transposed turn."""
    freq, axis = rope_frequencies(axes, base, factor, ramp)
    first, second = rope_pairs(len(freq), interleaved)
    angle = np.asarray(positions, dtype=np.float64)[axis].T * freq           # [T, pairs]
    z = (x[..., first] + 1j * x[..., second]) * (magnitude * np.exp(1j * sign * angle))[:, None]
    y = np.array(x, dtype=np.float64)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def rope_reach(x, axes, interleaved, magnitude=1.0):
    """|a| + |b| of each element's pair (0 where nothing turns): what an
    error of a cosine or sine is multiplied by."""
    first, second = rope_pairs(sum(axes) // 2, interleaved)
    r = np.zeros_like(x)
    r[..., first] = r[..., second] = abs(magnitude) * (np.abs(x[..., first]) + np.abs(x[..., second]))
    return r


# ------------------------------------------------------------------ the cache
def gather(pages, row, length):
    """The first `length` tokens [length, Hk, d] behind a table row; pages
    [P, Hk, page, d]."""
    page = pages.shape[2]
    out = np.zeros((length, pages.shape[1], pages.shape[3]))
    for j in range(length):
        out[j] = pages[row[j // page], :, j % page]
    return out


def append(pages, table, lens, cu, rows):
    """pages with the packed new tokens rows [T, Hk, d] at the sequences' ends."""
    pages = pages.copy()
    page = pages.shape[2]
    for s in range(len(cu) - 1):
        n = cu[s + 1] - cu[s]
        for i in range(n):
            p = lens[s] - n + i
            pages[table[s][p // page], :, p % page] = rows[cu[s] + i]
    return pages


def attn_rows(q, k, v, pos, causal, window, scale):
    """One sequence and one head: q [n, d] at positions pos, k and v [L, d].
    Returns o, lse and sum_j p_j |v_j| (what a relative error of the
    probabilities can move the output by)."""
    j = np.arange(k.shape[0])[None]
    p = np.asarray(pos)[:, None]
    seen = np.ones((len(pos), k.shape[0]), dtype=bool)
    if causal:
        seen &= j <= p
    if window > 0:
        seen &= j > p - window
    with np.errstate(invalid="ignore"):
        s = np.where(seen, (q @ k.T) * scale, -np.inf)
    o, reach = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(len(pos), -np.inf)
    for i in range(len(pos)):
        if not seen[i].any():
            continue
        m = s[i][seen[i]].max()
        e = np.exp(s[i][seen[i]] - m)
        lse[i] = m + math.log(e.sum())
        w = e / e.sum()
        o[i] = w @ v[seen[i]]
        reach[i] = w @ np.abs(v[seen[i]])
    return o, lse, reach


def paged_attn(q, k_pages, v_pages, table, lens, cu, causal=True, window=0, scale=None):
    """q [Tq, H, d]; returns o [Tq, H, d], lse [H, Tq] and the reach of o."""
    nh, hd = q.shape[1:]
    group = nh // k_pages.shape[1]
    scale = 1.0 / math.sqrt(hd) if scale is None else scale
    o, reach = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((nh, q.shape[0]), -np.inf)
    for s in range(len(cu) - 1):
        a, b = cu[s], cu[s + 1]
        if a == b:
            continue
        k, v = gather(k_pages, table[s], lens[s]), gather(v_pages, table[s], lens[s])
        pos = lens[s] - (b - a) + np.arange(b - a)
        for h in range(nh):
            o[a:b, h], lse[h, a:b], reach[a:b, h] = attn_rows(q[a:b, h], k[:, h // group], v[:, h // group], pos,
                                                              causal, window, scale)
    return o, lse, reach


# ------------------------------------------------------------------ page operations
class Pages:
    """Tables as plain lists; `data` maps a page to what it holds."""

    def __init__(self, table, lens, refs, page, data=None):
        self.table, self.lens, self.refs = [list(r) for r in table], list(lens), list(refs)
        self.page = page
        self.data = list(data) if data is not None else list(range(len(refs)))

    def used(self, n):
        return -(-n // self.page)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, counts):
        need = [self.used(n + c) - self.used(n) for n, c in zip(self.lens, counts)]
        if min(counts) < 0 or any(self.used(n + c) > len(self.table[0]) for n, c in zip(self.lens, counts)):
            return -1
        if any(c > 0 and n % self.page and self.refs[row[n // self.page]] > 1
               for n, c, row in zip(self.lens, counts, self.table)):
            return -2
        free = self.free_pages()
        if sum(need) > len(free):
            return sum(need) - len(free)
        for s, c in enumerate(counts):
            for j in range(self.used(self.lens[s]), self.used(self.lens[s] + c)):
                p = free.pop(0)
                self.table[s][j] = p
                self.refs[p] = 1
            self.lens[s] += c
        return 0

    def fork(self, parents, children):
        slots = range(len(self.lens))
        if any(p not in slots or c not in slots or p == c for p, c in zip(parents, children)):
            return -1
        if len(set(children)) < len(children) or any(self.lens[c] for c in children):
            return -1
        free = self.free_pages()
        need = sum(self.lens[p] % self.page != 0 for p in parents)
        if need > len(free):
            return need - len(free)
        lens = list(self.lens)
        for p, c in zip(parents, children):
            full = lens[p] // self.page
            for j in range(full):
                self.table[c][j] = self.table[p][j]
                self.refs[self.table[p][j]] += 1
            if lens[p] % self.page:
                new = free.pop(0)
                self.data[new] = self.data[self.table[p][full]]
                self.table[c][full] = new
                self.refs[new] = 1
            self.lens[c] = lens[p]
        return 0

    def release(self, slots):
        for s in slots:
            for j in range(self.used(self.lens[s])):
                self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            self.lens[s] = 0

    def truncate(self, lens):
        for s, n in enumerate(lens):
            for j in range(self.used(n), self.used(self.lens[s])):
                self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            self.lens[s] = min(self.lens[s], n)

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        new = dict(zip(movers, holes))
        for a, b in new.items():
            self.data[b] = self.data[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, n in enumerate(self.lens):
            for j in range(self.used(n)):
                self.table[s][j] = new.get(self.table[s][j], self.table[s][j])
        return live
