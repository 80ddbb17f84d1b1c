"""Float64 oracle of the 4-bit form of a paged cache.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see attn_f64).  The definition written
out group by group and byte by byte: what a group of 32 columns is held as, the
bytes of a page's head, and the values that bytes stand for.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32


def step_byte(top):
    """The byte of the step of a group whose largest magnitude is `top`."""
    if not math.isfinite(top):
        return 255
    want = top / 7.0
    if want < 2.0 ** -14:
        return int(math.floor(want * 2.0 ** 17 + 0.5))
    e = math.floor(math.log2(want))
    m = int(math.floor(want / 2.0 ** (e - 3) + 0.5))          # 8 .. 16
    return min(8 * (e + 15) + (m - 8), 247)


def step_of(byte):
    e, m = byte >> 3, byte & 7
    if e == 31:
        return math.nan
    return (8 + m) / 8.0 * 2.0 ** (e - 15) if e else m / 8.0 * 2.0 ** -14


STEPS = np.array([step_of(b) for b in range(256)])


def quantise(x):
    """x [..., d]: codes c [..., d] (whole numbers) and step bytes [..., d / 32]."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, GROUP)
    finite = np.isfinite(g).all(-1)
    top = np.where(finite, np.abs(np.where(np.isfinite(g), g, 0.0)).max(-1), np.inf)
    byte = np.array([step_byte(t) for t in top.reshape(-1)], dtype=np.int64).reshape(top.shape)
    s = STEPS[byte][..., None]
    with np.errstate(all="ignore"):
        c = np.where((s > 0) & finite[..., None], np.clip(np.floor(g / s + 0.5), -8, 7), 0.0)
    return c.reshape(x.shape).astype(np.int64), byte


def values(codes, byte):
    s = np.repeat(STEPS[byte], GROUP, axis=-1)
    return codes * s


def place(j, d, keys):
    """Byte and nibble of column j in a token's codes."""
    groups = d // GROUP
    q, i = divmod(j, GROUP)
    if keys:            # word i / 8 of group q, at place (i / 8) * groups + q
        word, k = divmod(i, 8)
        return (word * groups + q) * 4 + k // 2, k % 2
    half, k = divmod(i, 4)
    return (half * groups + q) * 2 + k // 2, k % 2


def pack(codes, byte, keys):
    """Blocks [..., page * 17 d / 32] uint8 of codes [..., page, d]."""
    *lead, page, d = codes.shape
    held = np.zeros((*lead, page, d // 2), dtype=np.uint8)
    for j in range(d):
        at, hi = place(j, d, keys)
        held[..., at] |= ((codes[..., j] + 8) << (4 * hi)).astype(np.uint8)
    return np.concatenate([held.reshape(*lead, -1), byte.astype(np.uint8).reshape(*lead, -1)], axis=-1)


def unpack(blocks, page, d, keys):
    """Codes [..., page, d] and step bytes [..., page, d / 32] of blocks."""
    *lead, _ = blocks.shape
    held = blocks[..., :page * d // 2].reshape(*lead, page, d // 2).astype(np.int64)
    byte = blocks[..., page * d // 2:].reshape(*lead, page, d // GROUP).astype(np.int64)
    codes = np.empty((*lead, page, d), dtype=np.int64)
    for j in range(d):
        at, hi = place(j, d, keys)
        codes[..., j] = ((held[..., at] >> (4 * hi)) & 15) - 8
    return codes, byte
