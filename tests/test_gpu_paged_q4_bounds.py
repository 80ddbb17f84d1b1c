"""The 4-bit paged cache at the ends of its numbers' range, against float64.

What a score may be off by (derived, for the arithmetic over codes): a group's sum
over its 32 columns begins at -8 sum q, a float32 sum of 32 numbers (off by 8 * 2^-24
of 8 sum|q| at most: five sums in a row), and two products of 16 columns add n q with
n <= 15.  No partial sum passes 23 sum|q|.  A product cuts each of its 17 addends, and
their sum, at 2^-23 of the largest at worst: 2 * 18 * 2^-23 * 23 sum|q| together.
Times the step, over the groups, with four roundings more of the row's sum (2^-21 of
each term), and the scale:

    E = scale sum_g s_g sum|q|_g (2 * 18 * 2^-23 * 23 + 64 * 2^-24 + 2^-21 * 8)

An LSE is off by the largest E of the row's keys and 2^-20 of itself (scale and
maximum in float32); each probability and their sum by that much of themselves too,
on top of 2^-8 for P's rounding (half a step, to bf16) and 2^-8 |o| for the output's.
"""
import numpy as np
import pytest
import torch

import mixed_length_dit_gb300 as zl
from oracle import paged_f64 as ref
from oracle import q4_f64 as q4
from _helpers import f64
from _q4 import BF16, Batch, pool_values

pytestmark = pytest.mark.gpu

E_SUM = 2 * 18 * 2.0 ** -23 * 23 + 64 * 2.0 ** -24 + 2.0 ** -21 * 8


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def rows_of(b, q, scale, causal=True, window=0):
    """For each (packed row, head): its scores over all keys of its sequence (-inf
    where hidden), what they may be off by, and the values [keys, d]."""
    kv, vv = pool_values(b.k_pages, True), pool_values(b.v_pages, False)
    steps = {}
    raw = b.k_pages.cpu().numpy()
    p, hk, page, row = raw.shape
    _, byte = q4.unpack(raw.reshape(p, hk, page * row), page, b.hd, True)
    held = q4.STEPS[byte]                                   # [P, Hk, page, d / 32]
    group = q.shape[1] // hk
    for s in range(len(b.new)):
        n, length = b.new[s], b.lens[s]
        k, v = ref.gather(kv, b.table[s], length), ref.gather(vv, b.table[s], length)
        st = ref.gather(held, b.table[s], length)
        j = np.arange(length)
        for i in range(n):
            pos = length - n + i
            seen = (j <= pos) if causal else np.ones(length, dtype=bool)
            if window:
                seen = seen & (j > pos - window)
            for h in range(q.shape[1]):
                x = q[b.cu[s] + i, h]
                score = np.where(seen, k[:, h // group] @ x * scale, -np.inf)
                off = st[:, h // group] @ np.abs(x).reshape(-1, 32).sum(-1) * scale * E_SUM
                yield b.cu[s] + i, h, score, np.where(seen, off, 0.0), v[:, h // group]


# ------------------------------------------------------------------ scores of any size
@pytest.mark.parametrize("exp", [12, 24, 29, 30, 31, 32, 40, 64, 100])
@pytest.mark.parametrize("new,lens,heads,kv_heads,hd,most", [
    ([1, 2], [200, 77], 8, 2, 128, 200),                    # units of 8 rows, whole
    ([1] * 3, [5000, 90, 1200], 4, 2, 64, 16000),           # cut
    ([4, 9], [900, 300], 8, 2, 128, 900),                   # units of 16 rows
    ([1], [3000], 2, 1, 64, 3000),                          # a cluster
])
def test_scores_of_any_size(new, lens, heads, kv_heads, hd, most, exp):
    """Scores of up to 2^100 and more: finite outputs, the lse to the scores' own
    rounding, and, where the largest score leads by more than the roundings of two
    scores and 60, the value of its key: a probability of one times a step is a bf16, and
    so is the value; the other keys together count for less than 2^-60."""
    b = Batch(new, lens, heads, kv_heads, hd, 16, seed=50, spare_cols=1000, scales=(2.0 ** exp, 1.0, 1.0))
    scale = hd ** -0.5
    o, lse = b.run(most=most)
    zl.sync_check()
    o, lse = f64(o), f64(lse)
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    clear = 0
    for row, h, score, off, v in rows_of(b, f64(b.q), scale):
        top = int(score.argmax())
        m = score[top]
        want = m + np.log(np.exp(score - m).sum())
        assert abs(lse[h, row] - want) <= off.max() + 2.0 ** -20 * abs(want)
        second = np.partition(score, -2)[-2] if len(score) > 1 else -np.inf
        if m - second > 2 * (off.max() + 2.0 ** -22 * abs(m)) + 60:
            clear += 1
            assert np.abs(o[row, h] - v[top]).max() <= 2.0 ** -60, (row, h)
    assert exp < 24 or clear >= 0.8 * o.shape[0] * o.shape[1]


def test_scores_of_a_chunk_up_to_their_bound():
    """Chunks run over the bf16 kernel, whose probabilities keep the rounding of the scaled
    maximum, below 2^7 in the exponent for scores below 2^30: finite, and the lse to the
    scores' rounding (twice the bound above: eight products of 16 columns, partial sums
    below 7 sum_g s_g sum|q|_g, 8 * 18 * 2^-23 * 7)."""
    b = Batch([100, 70], [300, 90], 2, 2, 128, 16, seed=49, scales=(2.0 ** 27, 1.0, 1.0))
    o, lse = b.run()
    zl.sync_check()
    o, lse = f64(o), f64(lse)
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    for row, h, score, off, v in rows_of(b, f64(b.q), 128 ** -0.5):
        assert score.max() < 2.0 ** 30
        want = score.max() + np.log(np.exp(score - score.max()).sum())
        assert abs(lse[h, row] - want) <= 2 * off.max() + 2.0 ** -20 * abs(want)


# ------------------------------------------------------------------ queries of any size
@pytest.mark.parametrize("exp", [100, 113, 115, 120, 125])
@pytest.mark.parametrize("new,lens,heads,kv_heads,hd,most", [
    ([1, 2], [200, 77], 8, 2, 128, 200), ([1] * 3, [5000, 90, 1200], 4, 2, 64, 16000), ([4, 9], [900, 300], 8, 2, 128, 900),
])
def test_queries_up_to_the_largest(new, lens, heads, kv_heads, hd, most, exp):
    """Queries near the end of bf16's range, two rows at the largest number itself (its
    columns' sum does not fit a float32), and a scale that makes the scores ordinary."""
    b = Batch(new, lens, heads, kv_heads, hd, 16, seed=51, spare_cols=1000, scales=(2.0 ** exp, 2.0 ** -10, 1.0))
    largest = float(torch.finfo(BF16).max)
    if exp == 125:
        b.q[0, 0] = largest
        b.q[-1, -1] = -largest
    scale = 2.0 ** (10 - exp) * hd ** -0.5
    o, lse = b.run(most=most, softmax_scale=scale)
    zl.sync_check()
    o, lse = f64(o), f64(lse)
    for row, h, score, off, v in rows_of(b, f64(b.q), scale):
        m = score.max()
        p = np.exp(score - m)
        want = m + np.log(p.sum())
        assert abs(lse[h, row] - want) <= off.max() + 2.0 ** -20 * max(abs(want), 1), (row, h, lse[h, row], want)
        p /= p.sum()
        reach, out = p @ np.abs(v), p @ v
        assert np.all(np.abs(o[row, h] - out) <= (2.0 ** -8 + 2 * off.max() + 2.0 ** -19) * reach + 2.0 ** -8 * np.abs(out))


@pytest.mark.parametrize("hd", [64, 128])
def test_large_queries_at_a_scale_of_one(hd):
    """A scale that is not small, and keys of which some read as zero: no infinity
    times zero comes in, and a row whose keys are all zero is their mean."""
    b = Batch([2, 3], [90, 40], 4, 2, hd, 16, seed=52, scales=(2.0 ** 122, 2.0 ** -12, 1.0))
    page = b.k_pages.shape[2]
    for s in (0, 1):                                        # the first sequence's first page, all of the second
        for p in b.table[s, :1 if s == 0 else 3]:
            b.k_pages[int(p)].view(2, -1)[:, page * hd // 2:] = 0
    o, lse = b.run(softmax_scale=1.0)
    zl.sync_check()
    o, lse = f64(o), f64(lse)
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    for row, h, score, off, v in rows_of(b, f64(b.q), 1.0):
        if row >= b.cu[1]:
            n = int(np.isfinite(score).sum())
            assert abs(lse[h, row] - np.log(n)) <= 2.0 ** -20 * np.log(n)
            reach = np.abs(v[:n]).mean(0)
            assert np.all(np.abs(o[row, h] - v[:n].mean(0)) <= 2.0 ** -8 * np.abs(v[:n].mean(0)) + 2.0 ** -19 * reach)
        else:
            assert abs(lse[h, row] - score.max()) <= off.max() + 2.0 ** -20 * abs(score.max()) + np.log(90)


# ------------------------------------------------------------------ what the pages hold
def pool_bytes(pool, b, rows, keys):
    """A pool's bytes once rows [T, Hk, d] are the sequences' last tokens."""
    raw = pool.cpu().numpy().copy()
    p, hk, page, row = raw.shape
    d = row * 32 // 17
    flat = raw.reshape(p, hk, page * row)
    codes, byte = q4.quantise(rows)
    for s in range(len(b.new)):
        for i in range(b.new[s]):
            pos = b.lens[s] - b.new[s] + i
            to, at = flat[b.table[s][pos // page]], pos % page
            block = q4.pack(codes[b.cu[s] + i][:, None], byte[b.cu[s] + i][:, None], keys)
            to[:, at * d // 2:(at + 1) * d // 2] = block[:, :d // 2]
            to[:, page * d // 2 + at * d // 32:page * d // 2 + (at + 1) * d // 32] = block[:, d // 2:]
    return raw


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("-nan"), float("inf"), float("-inf")])
def test_the_bytes_of_groups_that_are_not_finite(value, hd):
    """Their step is 255 and their codes are all zero (8 in the nibbles), whatever
    else they hold."""
    k = randn(53, 6, 2, hd)
    k[0, 0, 3], k[1, 1, 40], k[2, 0, hd - 1] = value, value, value
    k[3, 0, :32], k[4, 1, 32:64], k[5] = value, value, value
    k[4, 0, 7], k[4, 0, 9] = value, -value
    b = Batch([6], [20], 2, 2, hd, 16, seed=54)
    want = pool_bytes(b.k_pages, b, f64(k), True), pool_bytes(b.v_pages, b, f64(k), False)
    zl.paged_append_q4(k, k, *b.cache, b.cu)
    zl.sync_check()
    assert np.array_equal(b.k_pages.cpu().numpy(), want[0]) and np.array_equal(b.v_pages.cpu().numpy(), want[1])


@pytest.mark.parametrize("hd,heads,kv_heads,page,kw", [
    (64, 4, 2, 16, {}), (128, 10, 2, 64, {"interleaved": True}), (128, 3, 3, 256, {"axes": (64,)}),
    (64, 2, 1, 32, {"axes": (6,), "interleaved": True}), (128, 2, 1, 16, {"axes": (96,)}), (64, 3, 1, 16, {"axes": (6,)}),
    (128, 1, 1, 16, {"axes": (128,), "magnitude": 1.25}), (128, 2, 2, 16, {"axes": (70,), "interleaved": True}),
    (64, 1, 1, 16, {"axes": (62,)}), (128, 6, 2, 16, {"axes": (44, 42, 42)}), (64, 2, 2, 16, {"axes": (32,), "interleaved": True}),
    (128, 2, 2, 16, {"axes": (40, 24, 32), "interleaved": True, "magnitude": 0.75}), (64, 4, 4, 16, {"axes": (32, 16, 16)}),
])
def test_turned_keys_are_those_of_the_bf16_cache(hd, heads, kv_heads, page, kw):
    """The same bits: queries as paged_append and rope_fwd turn them, and the pages'
    bytes those of the keys that they turn."""
    b = Batch([1, 40, 0, 130, 300], [90, 40, 5, 333, 559], heads, kv_heads, hd, page, seed=55)
    c = Batch([1, 40, 0, 130, 300], [90, 40, 5, 333, 559], heads, kv_heads, hd, page, seed=55)
    k, v = randn(56, b.cu[-1], kv_heads, hd), randn(57, b.cu[-1], kv_heads, hd)
    plan, axes = zl.RopePlan(hd, **kw), len(kw.get("axes", (hd,)))
    pos = np.concatenate([np.arange(n - m, n) for m, n in zip(b.new, b.lens)]).astype(np.int32)
    pos = i32(pos) if axes == 1 else i32(np.stack([pos * (a + 3) % 777 for a in range(axes)]))
    given = {} if axes == 1 else {"positions": pos}
    q = zl.paged_append_q4(k, v, *b.cache, b.cu, q=b.q, rope=plan, **given)
    qt, kt = zl.rope_fwd(b.q, k, pos, plan)
    zl.paged_append_q4(kt, v, *c.cache, c.cu)
    pools = [torch.zeros((b.num_pages, kv_heads, page, hd), dtype=BF16, device="cuda") for _ in range(2)]
    qb = zl.paged_append(k, v, *pools, *b.cache[2:], b.cu, q=b.q, rope=plan, **given)
    zl.sync_check()
    assert torch.equal(qt, qb)
    assert torch.equal(q, qt), float((q != qt).float().mean())
    assert torch.equal(b.k_pages, c.k_pages) and torch.equal(b.v_pages, c.v_pages)


# ------------------------------------------------------------------ each key once
@pytest.mark.parametrize("new,lens,heads,kv_heads,hd,page,most", [
    ([1, 3, 1], [20011, 513, 6000], 8, 2, 128, 64, None), ([1, 3, 1], [20011, 513, 6000], 8, 2, 128, 16, 100000),
    ([1], [9001], 4, 1, 64, 32, None), ([1], [131], 40, 8, 128, 16, None), ([1] * 3, [3000, 1, 700], 3, 1, 128, 128, None),
    ([5, 2, 7], [4000, 333, 7011], 8, 4, 64, 16, None), ([9] * 4, [6001, 40, 2500, 8000], 4, 1, 128, 32, None),
    ([1] * 40, [100 + 53 * i for i in range(40)], 8, 8, 64, 16, 30000), ([3, 16, 1], [5000, 5000, 5000], 4, 4, 128, 256, None),
    ([33, 150], [3000, 2500], 2, 2, 128, 16, None),
])
def test_every_key_counts_once(new, lens, heads, kv_heads, hd, page, most):
    """Queries of zero: every key that is seen has the same probability, the lse is the
    logarithm of their number n (to 2^-17: logarithms below 16 in float32 are off by 2^-21,
    a part's, its weight's and the sum's add up to a few of them; a key more or less is
    1 / n), and as 32 keys have their values in one column and the next 32 in another, an
    output's columns say how many of their keys were counted (a probability of one times a
    step and the sums of sevens are exact: off by the last rounding, 2^-8, and 2^-17)."""
    b = Batch(new, lens, heads, kv_heads, hd, page, seed=58, spare_cols=3)
    if most is not None:
        b.dtable = torch.nn.functional.pad(b.dtable, (0, -(-most // page))).contiguous()
    b.q.zero_()
    rows = torch.zeros((sum(lens), kv_heads, hd), dtype=BF16)
    j = np.concatenate([np.arange(n) for n in lens])
    rows[torch.arange(len(j)), :, torch.tensor(j // 32 % hd)] = 7
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    zl.paged_append_q4(randn(60, *rows.shape), rows.cuda(), *b.cache, cu)
    for kw in ({}, {"window": 700}, {"causal": False}, {"window": 2049, "causal": False}):
        o, lse = b.run(most=most, **kw)
        zl.sync_check()
        o, lse = f64(o), f64(lse)
        for s, n in enumerate(new):
            for i in range(n):
                pos = lens[s] - n + i
                hi = pos + 1 if kw.get("causal", True) else lens[s]
                lo = max(0, pos - kw["window"] + 1) if "window" in kw else 0
                want = np.bincount(np.arange(lo, hi) // 32 % hd, minlength=hd) * 7 / (hi - lo)
                row = b.cu[s] + i
                assert np.abs(lse[:, row] - np.log(hi - lo)).max() <= 2.0 ** -17, (s, i, kw)
                assert np.all(np.abs(o[row] - want) <= (2.0 ** -8 + 2.0 ** -17) * want), (s, i, kw)


# ------------------------------------------------------------------ chunks in several batches
@pytest.mark.parametrize("heads,kv_heads,most,batches", [(16, 8, 131072, 4), (4, 2, 1100000, 7)])
def test_chunks_unpacked_batch_after_batch(heads, kv_heads, most, batches):
    """Seven chunks whose bound of the lengths lets the workspace hold two at a time,
    or one (a sequence of more than its 1 GiB), with single tokens and empty sequences
    between them.  (Scores of the bf16 products: eight of 16 columns, whose partial
    sums stay below 7 sum_g s_g sum|q|_g: 8 * 18 * 2^-23 * 7, below twice the bound above.)"""
    new = [1, 70, 0, 129, 2, 90, 200, 0, 65, 1, 100, 300, 1]
    lens = [300, 70, 9, 140, 600, 350, 201, 0, 500, 1, 90, 310, 77]
    b = Batch(new, lens, heads, kv_heads, 128, 256, seed=59)
    b.dtable = torch.nn.functional.pad(b.dtable, (0, most // 256 + 1 - b.dtable.shape[1]), value=-1).contiguous()
    for kw in ({}, {"causal": False}):
        zl.profile_begin()
        o, lse = b.run(most=most, **kw)
        names = zl.profile_end()
        zl.sync_check()
        assert names["paged_unpack_q4"][0] == batches, names
        o, lse = f64(o), f64(lse)
        for row, h, score, off, v in rows_of(b, f64(b.q), 128 ** -0.5, **kw):
            if not np.isfinite(score).any():
                assert np.isneginf(lse[h, row]) and np.all(o[row, h] == 0)
                continue
            off = 2 * off
            m = score.max()
            p = np.exp(score - m)
            want = m + np.log(p.sum())
            assert abs(lse[h, row] - want) <= off.max() + 2.0 ** -20 * max(abs(want), 1)
            p /= p.sum()
            reach, out = p @ np.abs(v), p @ v
            assert np.all(np.abs(o[row, h] - out) <= (2.0 ** -8 + 2 * off.max() + 2.0 ** -19) * reach + 2.0 ** -8 * np.abs(out))


# ------------------------------------------------------------------ ordinary scores
@pytest.mark.parametrize("new,lens,heads,kv_heads,hd,page,kw", [
    ([1, 3, 1], [20011, 513, 6000], 8, 2, 128, 64, {}), ([1, 3, 1], [20011, 513, 6000], 8, 2, 128, 16, {"window": 4097}),
    ([1] * 4, [1001, 33, 1, 700], 10, 2, 64, 16, {}), ([12, 40], [3000, 60], 4, 4, 128, 32, {"causal": False}),
    ([7, 3], [4100, 9000], 32, 8, 128, 32, {"window": 4096}),
])
def test_outputs_to_the_bound_of_their_arithmetic(new, lens, heads, kv_heads, hd, page, kw):
    """The bounds above for queries over codes, with steps as they come (some 20 times
    below what products of codes with 128 added would be allowed)."""
    b = Batch(new, lens, heads, kv_heads, hd, page, seed=61)
    o, lse = b.run(**kw)
    zl.sync_check()
    o, lse = f64(o), f64(lse)
    for row, h, score, off, v in rows_of(b, f64(b.q), hd ** -0.5, **kw):
        m = score.max()
        p = np.exp(score - m)
        want = m + np.log(p.sum())
        p /= p.sum()
        err = p @ off
        assert abs(lse[h, row] - want) <= err + 2.0 ** -20 * max(abs(want), 8), (row, h)
        reach, out = p @ np.abs(v), p @ v
        tol = (2.0 ** -8 + 2 * off.max() + 2.0 ** -19) * reach + 2.0 ** -8 * np.abs(out)
        assert np.all(np.abs(o[row, h] - out) <= tol), (row, h)
