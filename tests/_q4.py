"""Batches over a 4-bit cache for the tests (the bytes are the oracle's)."""
from __future__ import annotations

import numpy as np
import torch

import mixed_length_dit_gb300 as zl
from oracle import q4_f64 as q4

BF16 = torch.bfloat16


def pool_values(pool, keys):
    """The float64 values [P, Hk, page, d] that a pool's bytes stand for."""
    raw = pool.cpu().numpy()
    p, hk, page, row = raw.shape
    codes, byte = q4.unpack(raw.reshape(p, hk, page * row), page, row * 32 // 17, keys)
    with np.errstate(invalid="ignore"):
        return q4.values(codes, byte)


def random_pool(rng, pages, kv_heads, page, hd, keys, scale=1.0):
    """Bytes of random values whose size differs from group to group."""
    x = rng.standard_normal((pages, kv_heads, page, hd)) * scale
    x *= np.repeat(np.exp2(rng.integers(-2, 2, (pages, kv_heads, page, hd // 32))), 32, -1)
    codes, byte = q4.quantise(x)
    return torch.tensor(q4.pack(codes, byte, keys).reshape(pages, kv_heads, page, hd * 17 // 32))


class Batch:
    """New tokens and a 4-bit cache in use: pages in any order; pool rows and
    table entries that belong to nobody hold what must not matter."""

    def __init__(self, new, lens, heads, kv_heads, hd, page, seed=0, spare_cols=2, fill=0xff, device="cuda",
                 scales=(1.0, 1.0, 1.0)):
        rng = np.random.default_rng(seed)
        self.new, self.lens, self.hd, self.page, self.kv_heads = list(new), list(lens), hd, page, kv_heads
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        used = [-(-n // page) for n in lens]
        self.num_pages = sum(used) + 3
        numbers = rng.permutation(self.num_pages)
        cols = max(used) + spare_cols
        self.table = np.full((len(lens), cols), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(used):
            self.table[s, :n] = numbers[at:at + n]
            self.table[s, n:] = rng.integers(-5, self.num_pages + 5, cols - n)      # past the sequence: anything
            at += n
        self.k_pages, self.v_pages = (random_pool(rng, self.num_pages, kv_heads, page, hd, k, x)
                                      for k, x in ((True, scales[1]), (False, scales[2])))
        for pool in (self.k_pages, self.v_pages):
            for s, n in enumerate(lens):
                if n % page:
                    self.fill(pool, int(self.table[s, n // page]), n % page, fill)
            for p in numbers[at:]:
                self.fill(pool, int(p), 0, fill)
        self.k_pages, self.v_pages = self.k_pages.to(device), self.v_pages.to(device)
        self.q = torch.tensor(rng.standard_normal((self.cu[-1], heads, hd)) * scales[0], dtype=BF16, device=device)
        self.dtable = torch.tensor(self.table, device=device)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=device)

    def fill(self, pool, p, row, byte):
        """The bytes of the rows from `row` on, in every head of page p."""
        hd = self.hd
        flat = pool[p].view(self.kv_heads, -1)
        flat[:, row * hd // 2:self.page * hd // 2] = byte
        flat[:, self.page * hd // 2 + row * hd // 32:] = byte

    @property
    def cache(self):
        return self.k_pages, self.v_pages, self.dtable, self.dlens

    def run(self, q=None, most=None, **kw):
        return zl.paged_attn_q4(self.q if q is None else q, *self.cache, self.cu,
                                max(self.lens) if most is None else most, **kw)
