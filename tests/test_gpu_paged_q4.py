"""The 4-bit paged cache on the GPU: appended bytes and values read back are the
oracle's exactly; attention against the float64 definition over the values held.

Tolerance of an attention output o with reach r = sum_j p_j |v_j| (derived, per
element): each probability, or its product with a value's step, is rounded to
bf16 once (2^-8 of it at most), so the sum is off by 2^-8 r; the result is
rounded once, 2^-8 |o|.  Scores: the tensor cores may multiply codes with 128
added, so that a group's sum runs up to 136 * 2 * sum|q_i| over its 32 columns
(26 for the N(0, 1) queries here, 7,000) and is rounded, or cut, four times at
2^-23 of that, times a step (below 2 with the inputs here, 0.4 as a rule) and
the scale; of the four groups one or two have a large step: below 1.2e-3 of a
score together, so a probability is off by 1.2e-3 and its share of the sum by
twice that, 2^-8.7: (2^-8 + 2^-8.7) r is under 2^-7.2 r, and an LSE by 1.2e-3.
"""
import numpy as np
import pytest
import torch

import mixed_length_dit_gb300 as zl
from mixed_length_dit_gb300 import _lib
from oracle import paged_f64 as ref
from oracle import q4_f64 as q4
from _helpers import f64
from _q4 import BF16, Batch, pool_values

pytestmark = pytest.mark.gpu

TOL_SCORE = 1.2e-3


def check(b, o, lse, q=None, **kw):
    want, want_lse, reach = ref.paged_attn(f64(b.q if q is None else q), pool_values(b.k_pages, True),
                                           pool_values(b.v_pages, False), b.table, b.lens, b.cu, **kw)
    tol = (2.0 ** -8 + 2 * TOL_SCORE) * reach + 2.0 ** -8 * np.abs(want)
    err = np.abs(f64(o) - want)
    assert np.all(err <= tol), float((err - tol).max())
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(f64(lse)), none)
    err = np.abs(f64(lse)[~none] - want_lse[~none])
    assert np.all(err <= TOL_SCORE + 2.0 ** -20 * np.abs(want_lse[~none])), float(err.max())


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def appended(pool, b, rows, keys):
    """The bytes of a pool once rows [T, Hk, d] are its sequences' last tokens."""
    raw = pool.cpu().numpy().copy()
    p, hk, page, row = raw.shape
    d = row * 32 // 17
    flat = raw.reshape(p, hk, page * row)
    codes, byte = q4.quantise(rows)
    for s in range(len(b.cu) - 1):
        n = b.cu[s + 1] - b.cu[s]
        for i in range(n):
            pos = b.lens[s] - n + i
            to = flat[b.table[s][pos // page]]
            block = q4.pack(codes[b.cu[s] + i][:, None], byte[b.cu[s] + i][:, None], keys)
            at = pos % page
            to[:, at * d // 2:(at + 1) * d // 2] = block[:, :d // 2]
            to[:, page * d // 2 + at * d // 32:page * d // 2 + (at + 1) * d // 32] = block[:, d // 2:]
    return raw


# ------------------------------------------------------------------ append and read
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kv_heads,page", [(1, 16), (3, 32), (8, 64), (2, 256)])
def test_append_writes_the_oracles_bytes(kv_heads, page, hd):
    b = Batch([1, 40, 0, 130, 3], [90, 40, 5, 333, 259], kv_heads, kv_heads, hd, page, seed=1, fill=0x5a)
    rows = randn(2, b.cu[-1], 2 * kv_heads + 1, hd)             # keys and values of wider rows
    rows *= torch.exp2(torch.randint(-9, 9, (b.cu[-1], 2 * kv_heads + 1, 1), device="cuda")).to(BF16)
    k, v = rows[:, :kv_heads], rows[:, kv_heads:2 * kv_heads]
    want = appended(b.k_pages, b, f64(k), True), appended(b.v_pages, b, f64(v), False)
    assert zl.paged_append_q4(k, v, *b.cache, b.cu) is None
    zl.sync_check()
    assert np.array_equal(b.k_pages.cpu().numpy(), want[0]) and np.array_equal(b.v_pages.cpu().numpy(), want[1])
    kr, vr = zl.paged_read_q4(*b.cache, b.cu)
    zl.sync_check()
    assert np.array_equal(f64(kr), q4.values(*q4.quantise(f64(k)))) and np.array_equal(f64(vr), q4.values(*q4.quantise(f64(v))))


@pytest.mark.parametrize("hd", [64, 128])
def test_every_bf16_beside_every_largest_one(hd):
    """Codes and steps for all magnitudes of a group's largest value with eight
    bits, each with all values below it on a fine grid (halves among them)."""
    tops = [(128 + a) * 2.0 ** e for e in (-30, -26, -25, -24, -23, -22, -21, -20, -8, 0, 9, 11, 12, 90, 119) for a in range(128)]
    x = np.zeros((len(tops), 1, hd))
    rng = np.random.default_rng(3)
    for i, t in enumerate(tops):
        x[i, 0] = t * rng.integers(-256, 257, hd) / 256
        x[i, 0, 5] = -t
        s = q4.step_of(q4.step_byte(t))
        x[i, 0, 8:23] = np.minimum((np.arange(15) - 7.5) * s, t)
    k = torch.tensor(x).to(BF16).cuda()
    page = 256
    pools = [torch.zeros((8, 1, page, zl.q4_row_bytes(hd)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    cache = (*pools, table, i32([len(tops)]))
    zl.paged_append_q4(k, -k, *cache, [0, len(tops)])
    kr, vr = zl.paged_read_q4(*cache, [0, len(tops)])
    zl.sync_check()
    assert np.array_equal(f64(kr), q4.values(*q4.quantise(f64(k)))) and np.array_equal(f64(vr), q4.values(*q4.quantise(f64(-k))))


def test_what_is_not_finite_takes_its_group_along():
    k = randn(4, 6, 2, 128)
    k[0, 0, 3], k[1, 1, 40], k[2, 0, 127] = float("nan"), float("inf"), float("-inf")
    k[3] = 0
    k[4] = 3.3e38
    k[5] = 1e-30
    b = Batch([6], [20], 2, 2, 128, 16, seed=5)
    zl.paged_append_q4(k, k, *b.cache, b.cu)
    kr, vr = zl.paged_read_q4(*b.cache, b.cu)
    zl.sync_check()
    want = q4.values(*q4.quantise(f64(k)))
    assert np.array_equal(f64(kr), want, equal_nan=True) and np.array_equal(f64(vr), want, equal_nan=True)
    assert int(kr.isnan().sum()) == 3 * 32 and torch.all(kr[3] == 0) and torch.all(kr[5] == 0) and torch.all(kr[4] == 7 * 61440)


@pytest.mark.parametrize("hd,heads,kv_heads,page,kw", [
    (64, 4, 2, 16, {}), (128, 10, 2, 64, {"interleaved": True}), (128, 3, 3, 256, {"axes": (64,)}),
    (64, 2, 1, 32, {"axes": (6,), "interleaved": True}), (128, 2, 1, 16, {"axes": (96,)}), (64, 3, 1, 16, {"axes": (6,)}),
    (128, 1, 1, 16, {"axes": (128,), "magnitude": 1.25}), (128, 2, 2, 16, {"axes": (70,), "interleaved": True}),
    (64, 1, 1, 16, {"axes": (62,)}),
])
def test_append_turns_keys_and_queries(hd, heads, kv_heads, page, kw):
    b = Batch([1, 40, 0, 130, 3], [90, 40, 5, 333, 259], heads, kv_heads, hd, page, seed=6)
    k, v = randn(7, b.cu[-1], kv_heads, hd), randn(8, b.cu[-1], kv_heads, hd)
    plan, axes, il, m = zl.RopePlan(hd, **kw), kw.get("axes", (hd,)), kw.get("interleaved", False), kw.get("magnitude", 1.0)
    pos = np.concatenate([np.arange(n - c, n) for c, n in zip(b.new, b.lens)])[None]
    for inplace in (False, True):
        queries = b.q.clone()
        q = zl.paged_append_q4(k, v, *b.cache, b.cu, q=queries, rope=plan, q_out=queries if inplace else None)
        kr, vr = zl.paged_read_q4(*b.cache, b.cu)
        zl.sync_check()
        want = ref.rope(f64(b.q), pos, axes, interleaved=il, magnitude=m)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * ref.rope_reach(f64(b.q), axes, il, m)
        assert np.all(np.abs(f64(q) - want) <= tol)
        assert np.array_equal(f64(vr), q4.values(*q4.quantise(f64(v))))
        # a key is rounded to bf16, then to the nearest code of a step that is the largest one's seventh to 1/16
        want = ref.rope(f64(k), pos, axes, interleaved=il, magnitude=m)
        off = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * ref.rope_reach(f64(k), axes, il, m)
        top = np.abs(want).reshape(*want.shape[:2], -1, 32).max(-1) * (1 + 2.0 ** -7)
        step = np.repeat(top / 7 * (1 + 1 / 16), 32, -1)
        assert np.all(np.abs(f64(kr) - want) <= step / 2 + off)


def test_append_with_positions_of_three_axes():
    b = Batch([5, 30], [20, 300], 4, 2, 128, 16, seed=9)
    k, v = randn(10, 35, 2, 128), randn(11, 35, 2, 128)
    plan = zl.RopePlan(128, axes=(44, 42, 42))
    pos = torch.randint(0, 500, (3, 35), dtype=torch.int32, device="cuda")
    q = zl.paged_append_q4(k, v, *b.cache, b.cu, q=b.q, rope=plan, positions=pos)
    kr, vr = zl.paged_read_q4(*b.cache, b.cu)
    zl.sync_check()
    want = ref.rope(f64(b.q), pos.cpu().numpy(), (44, 42, 42))
    assert np.all(np.abs(f64(q) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * ref.rope_reach(f64(b.q), (44, 42, 42), False))
    turned, _ = zl.rope_fwd(k, None, pos, plan)
    held = q4.values(*q4.quantise(f64(turned)))
    # the same keys but for a bf16 here and there that the two kernels' sums round apart
    assert np.mean(f64(kr) != held) < 0.01 and np.array_equal(f64(vr), q4.values(*q4.quantise(f64(v))))


def test_append_outside_the_cache_is_left_out_and_reported():
    b = Batch([3, 2], [30, 20], 2, 1, 64, 16, seed=12)
    k = randn(13, 5, 1, 64)
    before = b.k_pages.clone(), b.v_pages.clone()
    for lens, entry in (([10 ** 6, 20], -1), ([30, 20], b.num_pages), ([2 ** 31 - 1, -5], 0)):
        b.dlens.copy_(i32(lens))
        b.dtable.copy_(torch.tensor(b.table))
        b.dtable[1, 1] = entry
        if lens[0] == 30:
            b.dtable[0] = -9
        zl.paged_append_q4(k, k, *b.cache, b.cu)
        with pytest.raises(zl.ZlError) as e:
            zl.sync_check()
        assert e.value.status == -8
        assert torch.equal(b.k_pages, before[0]) and torch.equal(b.v_pages, before[1])
        kr, vr = zl.paged_read_q4(*b.cache, b.cu)
        with pytest.raises(zl.ZlError):
            zl.sync_check()
        assert torch.all(kr == 0) and torch.all(vr == 0)
    b.dlens.copy_(i32([1, 20]))            # shorter than the new tokens: the last of them is its only one
    b.dtable.copy_(torch.tensor(b.table))
    zl.paged_append_q4(k, k, *b.cache, b.cu)
    with pytest.raises(zl.ZlError):
        zl.sync_check()
    kr, _ = zl.paged_read_q4(*b.cache, b.cu)
    with pytest.raises(zl.ZlError):
        zl.sync_check()
    assert torch.all(kr[:2] == 0) and np.array_equal(f64(kr[2:]), q4.values(*q4.quantise(f64(k[2:]))))


@pytest.mark.parametrize("way", ["short", "stream"])
def test_append_behind_a_refused_extend_writes_nothing(way):
    b = Batch([3, 20], [30, 50], 2, 2, 128, 16, seed=14)
    k = randn(15, 23, 2, 128)
    kw = {"stream": torch.cuda.Stream()} if way == "stream" else {}
    before = b.k_pages.clone()
    torch.cuda.synchronize()
    q = zl.paged_append_q4(k, k, *b.cache, b.cu, q=b.q, status=i32([4]), **kw)
    with pytest.raises(zl.ZlError):
        zl.sync_check(**kw)
    assert torch.equal(b.k_pages, before) and torch.equal(q, b.q)
    torch.cuda.synchronize()
    zl.paged_append_q4(k, k, *b.cache, b.cu, status=i32([0]), **kw)
    torch.cuda.synchronize()
    zl.sync_check()
    assert np.array_equal(b.k_pages.cpu().numpy(), appended(before, b, f64(k), True))


def test_read_into_wider_rows():
    b = Batch([7, 300], [50, 300], 2, 2, 64, 32, seed=16)
    k, v = zl.paged_read_q4(*b.cache, b.cu)
    rows = torch.full((b.cu[-1], 6, 64), 9.0, dtype=BF16, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    k2, v2 = zl.paged_read_q4(*b.cache, b.cu, k_out=rows[:, 1:3], v_out=rows[:, 4:], stream=stream)
    torch.cuda.synchronize()
    zl.sync_check()
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.all(rows[:, 0] == 9) and torch.all(rows[:, 3] == 9)
    kv = pool_values(b.k_pages, True)
    want = np.concatenate([ref.gather(kv, b.table[s], b.lens[s])[-n:] for s, n in enumerate(b.new)])
    assert np.array_equal(f64(k), want)
    with pytest.raises(ValueError, match="overlap"):
        zl.paged_read_q4(*b.cache, b.cu, k_out=rows[:, 1:3], v_out=rows[:, 2:4])


@pytest.mark.parametrize("slots", [70, 1300])
def test_append_and_read_many_sequences(slots):
    rng = np.random.default_rng(17)
    lens = [int(x) for x in rng.integers(1, 60, slots)]
    new = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 4, slots))]
    b = Batch(new, lens, 1, 1, 64, 16, seed=17)
    k = randn(18, b.cu[-1], 1, 64)
    want = appended(b.k_pages, b, f64(k), True)
    zl.paged_append_q4(k, k, *b.cache, b.cu)
    kr, _ = zl.paged_read_q4(*b.cache, b.cu)
    zl.sync_check()
    assert np.array_equal(b.k_pages.cpu().numpy(), want) and np.array_equal(f64(kr), q4.values(*q4.quantise(f64(k))))


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 1), (10, 2), (6, 2), (40, 8)])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_single_tokens(heads, kv_heads, hd, page):
    b = Batch([1] * 8, [1, 2, 31, 32, 33, 128, 129, 700], heads, kv_heads, hd, page)
    o, lse = b.run()
    zl.sync_check()
    check(b, o, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,kv_heads,hd,page", [(2, 2, 64, 16), (6, 2, 128, 32), (10, 2, 128, 128), (7, 1, 64, 64)])
def test_chunks(heads, kv_heads, hd, page, causal):
    new = [130, 1, 300, 0, 37, 128, 2, 257, 9, 16, 4]
    lens = [130, 500, 431, 90, 300, 1000, 64, 258, 9, 17, 350]
    b = Batch(new, lens, heads, kv_heads, hd, page, seed=21)
    o, lse = b.run(causal=causal)
    zl.sync_check()
    check(b, o, lse, causal=causal)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 96, 127, 128, 129, 200])
def test_every_number_of_rows(rows, hd):
    b = Batch([rows, rows // 3 + 1], [rows + 211, 600], 2, 2, hd, 16, seed=22)
    for kw in ({}, {"causal": False}, {"window": 70}):
        o, lse = b.run(**kw)
        zl.sync_check()
        check(b, o, lse, **kw)


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 7), (True, 128), (True, 200), (False, 33), (False, 129),
                                           (True, 10 ** 6)])
def test_windows(causal, window):
    b = Batch([1, 260, 33, 5], [900, 500, 33, 389], 6, 2, 64, 32, seed=23)
    o, lse = b.run(causal=causal, window=window)
    zl.sync_check()
    check(b, o, lse, causal=causal, window=window)


@pytest.mark.parametrize("group", [3, 5, 7, 12, 48, 100, 128])
def test_many_heads_of_one_key_head(group):
    b = Batch([1, 9, 40], [300, 140, 44], group, 1, 64, 16, seed=24)
    o, lse = b.run()
    zl.sync_check()
    check(b, o, lse)


def test_long_caches_are_split_and_joined():
    b = Batch([1, 3, 1], [20011, 513, 6000], 8, 2, 128, 64, seed=25)
    for kw in ({}, {"window": 4097}, {"causal": False}):
        o, lse = b.run(**kw)
        zl.sync_check()
        check(b, o, lse, **kw)
    o, lse = b.run(most=b.dtable.shape[1] * b.page)
    check(b, o, lse)


@pytest.mark.parametrize("new,lens,heads,kv_heads,hd", [
    ([1], [700], 8, 8, 64), ([1] * 19, [130] * 18 + [1000], 16, 8, 128), ([3, 1, 2], [3, 0, 600], 12, 4, 64),
    ([200], [600], 4, 4, 128), ([600, 129, 300], [620, 129, 1], 3, 1, 64), ([90, 1, 400, 2], [90, 500, 700, 7], 20, 4, 128),
    ([130] * 5, [0, 1, 200, 640, 64], 6, 2, 64), ([12, 5], [3000, 40], 4, 1, 128),
])
def test_the_bound_of_the_lengths_does_not_matter(new, lens, heads, kv_heads, hd):
    b = Batch(new, lens, heads, kv_heads, hd, 32, seed=26, spare_cols=2000)
    for kw in ({}, {"causal": False}, {"window": 100}):
        for most in (max(lens), 4000, 60000):
            o, lse = b.run(most=most, **kw)
            zl.sync_check()
            check(b, o, lse, **kw)


@pytest.mark.parametrize("slots", [70, 700])
def test_more_sequences_than_few_and_than_one_launch_holds(slots):
    rng = np.random.default_rng(27)
    new = [int(x) for x in rng.choice([0, 1, 1, 5, 40, 129, 140], slots)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 60, slots))]
    b = Batch(new, lens, 1, 1, 64, 16, seed=27)
    o, lse = b.run()
    zl.sync_check()
    check(b, o, lse)


def test_rows_that_see_nothing():
    """Lengths shorter than the chunk (positions below zero) and empty ones."""
    b = Batch([5, 3, 1, 200, 20], [2, 0, 0, 150, 7], 4, 2, 64, 16, seed=28)
    for kw in ({}, {"causal": False}, {"window": 2}):
        o, lse = b.run(**kw)
        zl.sync_check()
        check(b, o, lse, **kw)
        assert torch.isfinite(o.float()).all()
    assert torch.all(o[5:9] == 0)


def test_no_key_at_all():
    b = Batch([2, 200], [16, 16], 4, 2, 64, 16, seed=29)
    b.dlens.zero_()
    for most in (0, 16):
        o, lse = b.run(most=most)
        zl.sync_check()
        assert torch.all(o == 0) and torch.isneginf(lse).all()


@pytest.mark.parametrize("fill", [0xff, 0xf8, 0x00, 0xf7])
def test_what_belongs_to_nobody_does_not_matter(fill):
    b = Batch([1, 40, 200], [77, 100, 333], 4, 2, 128, 64, seed=30, fill=fill)
    o, lse = b.run()
    zl.sync_check()
    check(b, o, lse)


@pytest.mark.parametrize("new", [1, 20])
def test_windows_as_large_as_an_int(new):
    b = Batch([new, new], [10, 300], 4, 1, 64, 16, seed=31)
    for causal in (True, False):
        want = b.run(causal=causal)
        got = b.run(causal=causal, window=2 ** 31 - 1)
        zl.sync_check()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_large_scores():
    """Scores of thousands, whose running maximum jumps block by block: the lse to
    the scores' own rounding (64 times the inputs of the bound above, at a scale of
    one instead of 1/8: 512 times 1.2e-3), and the output that of the largest keys."""
    b = Batch([1, 50], [700, 700], 4, 2, 64, 16, seed=32)
    b.q *= 64
    o, lse = b.run(softmax_scale=1.0)
    zl.sync_check()
    want, want_lse, _ = ref.paged_attn(f64(b.q), pool_values(b.k_pages, True), pool_values(b.v_pages, False), b.table,
                                       b.lens, b.cu, scale=1.0)
    off = 512 * TOL_SCORE
    assert np.abs(f64(lse) - want_lse).max() <= off + 2.0 ** -20 * np.abs(want_lse).max()
    assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("q_exp,k_exp,v_exp", [(60, 0, 0), (-60, 0, 0), (110, -8, 10), (-120, 12, -12), (0, -12, 13), (0, 13, -13)])
@pytest.mark.parametrize("hd", [64, 128])
def test_large_and_small_numbers(q_exp, k_exp, v_exp, hd):
    """Queries, keys and values of other sizes, the scale making the scores what they
    were: the same tolerances (all but the roundings is a power of two), but for steps
    below 2^-14, whose units of 2^-17 the oracle has too."""
    b = Batch([1, 12, 30, 140], [500, 300, 77, 400], 4, 2, hd, 16, seed=39,
              scales=(2.0 ** q_exp, 2.0 ** k_exp, 2.0 ** v_exp))
    scale = 2.0 ** -(q_exp + k_exp) * hd ** -0.5
    o, lse = b.run(softmax_scale=scale)
    zl.sync_check()
    check(b, o, lse, scale=scale)


def test_steps_of_all_sizes_side_by_side():
    """Values whose steps differ by 2^30 from token to token: the small ones count
    where the large ones are not seen."""
    b = Batch([4, 1], [200, 200], 4, 2, 128, 16, seed=47)
    for pool, byte in ((b.v_pages, 0xf0), (b.k_pages, 0x08)):
        page = pool[int(b.table[0, 199 // 16])].view(2, -1)
        page[:, 16 * 64 + 199 % 16 * 4:16 * 64 + (199 % 16 + 1) * 4] = byte          # the newest token's steps
        page = pool[int(b.table[1, 3])].view(2, -1)
        page[:, 16 * 64:16 * 64 + 4 * 5] = 8 if byte == 0xf0 else 0
    o, lse = b.run()
    zl.sync_check()
    check(b, o, lse)


@pytest.mark.parametrize("new,lens,heads,kv_heads,hd", [
    ([1, 1], [40, 300], 8, 2, 128), ([12, 3], [200, 90], 10, 2, 64), ([100], [260], 1, 1, 128), ([300, 70], [300, 900], 4, 2, 64),
    ([1], [20000], 6, 2, 128), ([20], [9000], 2, 1, 64), ([5], [333], 8, 2, 128),
])
def test_nan_is_handed_on(new, lens, heads, kv_heads, hd):
    """A query or a visible key of NaN makes its rows NaN, as the formula does,
    and no other row's bits change."""
    b = Batch(new, lens, heads, kv_heads, hd, 16, seed=33)
    o1, l1 = b.run()
    q = b.q.clone()
    rows = [0, b.cu[-1] - 1]
    q[rows, heads - 1, 3] = float("nan")
    o2, l2 = b.run(q=q)
    nan = torch.zeros((b.cu[-1], heads), dtype=torch.bool, device="cuda")
    nan[rows, heads - 1] = True
    assert o2[nan].isnan().all() and l2.T[nan].isnan().all()
    assert torch.equal(o2[~nan], o1[~nan]) and torch.equal(l2.T[~nan], l1.T[~nan])
    # the last sequence's newest key: its last query alone sees it
    s, n = len(lens) - 1, lens[-1]
    step = 16 * hd // 2 + (n - 1) % 16 * hd // 32
    b.k_pages[int(b.table[s, (n - 1) // 16]), 0].view(-1)[step] = 0xff
    o3, l3 = b.run()
    zl.sync_check()
    nan[:] = False
    nan[-1, :heads // kv_heads] = True
    assert o3[nan].isnan().all() and l3.T[nan].isnan().all()
    assert torch.equal(o3[~nan], o1[~nan]) and torch.equal(l3.T[~nan], l1.T[~nan])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads,kv_heads,hd", [(4, 2, 64), (4, 4, 128)])
def test_a_query_that_is_not_finite_and_sees_no_key(heads, kv_heads, hd, value):
    """Such a row is zero and its lse -inf, as any row that sees nothing; one that
    sees keys is NaN."""
    new, lens = [1, 5, 9, 300], [0, 2, 40, 250]          # 3 queries, and 50, come before their cache
    b = Batch(new, lens, heads, kv_heads, hd, 16, seed=41)
    o1, l1 = b.run()
    q = b.q.clone()
    blind = [0, 1, 3, 15, 64]                            # rows of the packed batch that see nothing
    q[blind + [4, 10], 0, 5] = value
    o2, l2 = b.run(q=q)
    zl.sync_check()
    assert torch.all(o2[blind] == 0) and torch.isneginf(l2[:, blind]).all()
    assert o2[[4, 10], 0].isnan().all() and l2[0, [4, 10]].isnan().all()
    hit = torch.zeros((b.cu[-1], heads), dtype=torch.bool, device="cuda")
    hit[[4, 10], 0] = True
    assert torch.equal(o2[~hit], o1[~hit]) and torch.equal(l2.T[~hit], l1.T[~hit])


def test_queries_inside_wider_rows_and_given_buffers():
    b = Batch([1, 200, 7], [50, 260, 130], 6, 2, 128, 32, seed=34)
    o1, l1 = b.run()
    rows = randn(35, b.cu[-1], 10, 128)
    rows[:, 2:8] = b.q
    out, lse = torch.full_like(o1, 9.0), torch.full_like(l1, 9.0)
    ws = zl.alloc_workspace(zl.paged_attn_q4_workspace_bytes(b.cu, max(b.lens), 6, 2, 128), "cuda")
    ws.fill_(0xff)
    o2, l2 = b.run(q=rows[:, 2:8], out=out, lse=lse, workspace=ws)
    assert o2 is out and l2 is lse and torch.equal(o1, out) and torch.equal(l1, lse)
    with pytest.raises(zl.ZlError) as e:
        b.run(workspace=ws[:-16])
    assert e.value.status == _lib.ZL_EWORKSPACE


def test_same_bits_every_time():
    b = Batch([1, 300, 2, 11], [5000, 900, 2500, 700], 8, 2, 128, 16, seed=36)
    o, lse = b.run()
    for _ in range(5):
        o2, l2 = b.run()
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_pages_and_lengths_out_of_range_are_left_out_and_reported():
    b = Batch([1, 1, 4, 140], [100, 90, 60, 200], 4, 2, 64, 16, seed=37)
    for row, col, entry in ((1, 2, b.num_pages), (1, 2, -7), (3, 4, 1 << 30)):
        b.dtable[row, col] = entry
        b.run()
        with pytest.raises(zl.ZlError) as e:
            zl.sync_check()
        assert e.value.status == -8
        b.dtable.copy_(torch.tensor(b.table))
    for row in (1, 3):
        for n in (5000, -3):
            b.dlens[row] = n
            b.run()
            with pytest.raises(zl.ZlError):
                zl.sync_check()
        b.dlens[row] = b.lens[row]
    o, lse = b.run()
    zl.sync_check()
    check(b, o, lse)


def test_graph_replays_with_the_lengths_and_pages_of_the_moment():
    b = Batch([1, 1, 1, 150], [40, 2500, 333, 500], 8, 2, 128, 16, seed=38, spare_cols=6)
    most = b.dtable.shape[1] * 16
    out, lse = torch.zeros_like(b.q), torch.zeros((8, b.cu[-1]), device="cuda")
    ws = zl.alloc_workspace(zl.paged_attn_q4_workspace_bytes(b.cu, most, 8, 2, 128), "cuda")
    b.run(most=most, out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(most=most, out=out, lse=lse, workspace=ws)
    for lens in ([40, 2500, 333, 500], [33, 17, 330, 160], [1, 1290, 16, 499]):
        b.lens = lens
        b.dlens.copy_(i32(lens))
        g.replay()
        zl.sync_check()
        check(b, out, lse)


def test_two_streams_at_once_and_two_graphs_on_one_workspace():
    bs = [Batch([1, 90], [3000 + 500 * i, 300], 8, 2, 128, 16, seed=40 + i) for i in range(2)]
    want = [b.run() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    got = [b.run(stream=s) for _ in range(5) for b, s in zip(bs, streams)]
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    ws = zl.alloc_workspace(max(zl.paged_attn_q4_workspace_bytes(b.cu, max(b.lens), 8, 2, 128) for b in bs), "cuda")
    outs = [(torch.zeros_like(b.q), torch.zeros((8, b.cu[-1]), device="cuda")) for b in bs]
    graphs = []
    for b, (out, lse) in zip(bs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(out=out, lse=lse, workspace=ws)
        graphs.append(g)
    ws.fill_(255)                           # nothing of an earlier call is needed
    for i in (0, 1, 1, 0, 0, 1):
        for t in outs[i]:
            t.zero_()
        graphs[i].replay()
        zl.sync_check()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes, of which the last pages are used: the same
    bits as with a small pool."""
    small = Batch([1, 150, 4], [700, 400, 4], 16, 16, 128, 128, seed=42, fill=0)
    k, v = randn(43, 155, 16, 128), randn(44, 155, 16, 128)
    pages = 2 ** 32 // (16 * 128 * 68) + 40
    big = [torch.zeros((pages, 16, 128, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 32
    shift = pages - small.num_pages
    for x, y in zip(big, (small.k_pages, small.v_pages)):
        x[shift:] = y
    used = torch.arange(small.dtable.shape[1], device="cuda") < (small.dlens[:, None] + 127) // 128
    table = torch.where(used, small.dtable + shift, -1).int()
    zl.paged_append_q4(k, v, *small.cache, small.cu)
    zl.paged_append_q4(k, v, *big, table, small.dlens, small.cu)
    zl.sync_check()
    assert torch.equal(big[0][shift:], small.k_pages) and torch.equal(big[1][shift:], small.v_pages)
    for x, y in zip(zl.paged_read_q4(*small.cache, small.cu), zl.paged_read_q4(*big, table, small.dlens, small.cu)):
        assert torch.equal(x, y)
    o1, l1 = small.run()
    o2, l2 = zl.paged_attn_q4(small.q, *big, table, small.dlens, small.cu, 700)
    zl.sync_check()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


# ------------------------------------------------------------------ a run of them together
def test_generation_loop():
    """Prompts, single tokens, a fork, drafts taken back, a sequence freed and the
    pool compacted, on a 4-bit cache of two layers: every step's attention is that
    over the values that were held when they were appended."""
    layers, page, hd, heads, kv, slots, pages = 2, 16, 128, 6, 2, 6, 80
    g = torch.Generator(device="cuda").manual_seed(45)
    cache = torch.full((layers, 2, pages, kv, page, zl.q4_row_bytes(hd)), 0xff, dtype=torch.uint8, device="cuda")
    table = torch.full((slots, 24), -1, dtype=torch.int32, device="cuda")
    lens, refs = i32([0] * slots), i32([0] * pages)
    past = [[np.zeros((0, 2, kv, hd)) for _ in range(layers)] for _ in range(slots)]
    host = ref.Pages(table.tolist(), [0] * slots, [0] * pages, page)

    def step(counts):
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        status = zl.pages_extend(table, lens, refs, i32(counts), page)
        assert host.extend(counts) == 0
        for layer in range(layers):
            q = torch.randn((cu[-1], heads, hd), generator=g, device="cuda").to(BF16)
            k, v = (torch.randn((cu[-1], kv, hd), generator=g, device="cuda").to(BF16) for _ in range(2))
            held = cache[layer, 0], cache[layer, 1], table, lens
            zl.paged_append_q4(k, v, *held, cu, status=status)
            o, lse = zl.paged_attn_q4(q, *held, cu, 24 * page)
            zl.sync_check()
            new = np.stack([q4.values(*q4.quantise(f64(x))) for x in (k, v)], 1)
            for s in range(slots):
                if counts[s] == 0:
                    continue
                past[s][layer] = np.concatenate([past[s][layer], new[cu[s]:cu[s + 1]]])
                n = past[s][layer].shape[0]
                assert n == host.lens[s]
                for h in range(heads):
                    kk, vv = past[s][layer][:, 0, h // 3], past[s][layer][:, 1, h // 3]
                    want, wl, reach = ref.attn_rows(f64(q)[cu[s]:cu[s + 1], h], kk, vv, n - counts[s] + np.arange(counts[s]),
                                                    True, 0, hd ** -0.5)
                    err = np.abs(f64(o)[cu[s]:cu[s + 1], h] - want)
                    assert np.all(err <= (2.0 ** -8 + 2 * TOL_SCORE) * reach + 2.0 ** -8 * np.abs(want))
                    assert np.all(np.abs(f64(lse)[h, cu[s]:cu[s + 1]] - wl) <= TOL_SCORE + 2.0 ** -20 * np.abs(wl))

    step([35, 200, 16, 0, 0, 0])
    step([1, 1, 1, 0, 0, 0])
    assert int(zl.pages_fork(cache, table, lens, refs, i32([1, 1, 2]), i32([3, 5, 4]))) == host.fork([1, 1, 2], [3, 5, 4]) == 0
    for p, c in ((1, 3), (1, 5), (2, 4)):
        past[c] = list(past[p])
    step([1, 1, 1, 1, 1, 1])
    step([0, 20, 5, 3, 0, 150])
    keep = [n - d for n, d in zip(host.lens, [0, 18, 3, 3, 0, 1])]
    zl.pages_truncate(table, lens, refs, i32(keep), page)
    host.truncate(keep)
    for s in range(slots):
        past[s] = [x[:keep[s]] for x in past[s]]
    zl.pages_free(table, lens, refs, i32([0, 3]), page)
    host.release([0, 3])
    for s in (0, 3):
        past[s] = [np.zeros((0, 2, kv, hd)) for _ in range(layers)]
    assert int(zl.pages_compact(cache, table, lens, refs)) == host.compact()
    assert refs.tolist() == host.refs and lens.tolist() == host.lens
    step([17, 1, 1, 0, 1, 2])
    # all of it read back at once
    cu = [0]
    for n in host.lens:
        cu.append(cu[-1] + n)
    for layer in range(layers):
        k, v = zl.paged_read_q4(cache[layer, 0], cache[layer, 1], table, lens, cu)
        zl.sync_check()
        for s in range(slots):
            assert np.array_equal(f64(k)[cu[s]:cu[s + 1]], past[s][layer][:, 0])
            assert np.array_equal(f64(v)[cu[s]:cu[s + 1]], past[s][layer][:, 1])


def test_a_captured_step_with_appends():
    """Extend, append and attention in one graph, replayed: as the calls one by one."""
    page, hd, heads, kv, slots = 16, 64, 8, 2, 5

    def setup():
        cache = torch.zeros((2, 60, kv, page, zl.q4_row_bytes(hd)), dtype=torch.uint8, device="cuda")
        return cache, torch.full((slots, 10), -1, dtype=torch.int32, device="cuda"), i32([0] * slots), i32([0] * 60)

    counts, cu = i32([3, 1, 0, 2, 1]), zl.host_int32([0, 3, 4, 4, 6, 7])
    q, k, v = (torch.empty((7, h, hd), dtype=BF16, device="cuda") for h in (heads, kv, kv))
    ws = zl.alloc_workspace(zl.paged_attn_q4_workspace_bytes(cu, 160, heads, kv, hd), "cuda")
    plan = zl.RopePlan(hd)

    def step(c):
        cache, table, lens, refs = c
        status = zl.pages_extend(table, lens, refs, counts, page)
        qr = zl.paged_append_q4(k, v, cache[0], cache[1], table, lens, cu, q=q, rope=plan, status=status)
        return zl.paged_attn_q4(qr, cache[0], cache[1], table, lens, cu, 160, workspace=ws)

    eager, graphed = setup(), setup()
    for x in (q, k, v):
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(graphed)
    for i in range(20):
        for j, x in enumerate((q, k, v)):
            x.copy_(randn(100 * j + i, *x.shape))
        want = step(eager)
        graph.replay()
        zl.sync_check()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert torch.equal(eager[0], graphed[0]) and eager[2].tolist() == [60, 20, 0, 40, 20]


def test_the_long_way_gives_the_same_bits(monkeypatch):
    """The compiled short way of the binding against the checks in Python."""
    class Long:
        def __getattr__(self, name):
            return lambda *args: None

    taken = []

    class Counting:
        real = _lib.bind()

        def __getattr__(self, name):
            def call(*args):
                r = getattr(self.real, name)(*args)
                if r is not None:
                    taken.append(name)
                return r
            return call

    results = []
    for binding in (Counting(), Long()):
        monkeypatch.setattr(_lib, "_bind", binding)
        b = Batch([1, 200, 7], [50, 260, 130], 6, 2, 128, 32, seed=46)
        k = randn(47, b.cu[-1], 2, 128)
        q = zl.paged_append_q4(k, -k, *b.cache, b.cu, q=b.q, rope=zl.RopePlan(128))
        results.append([q, *zl.paged_read_q4(*b.cache, b.cu), *b.run(q=q), b.k_pages, b.v_pages])
    assert taken == ["append_q4", "read_q4", "attn_q4"]
    zl.sync_check()
    assert all(torch.equal(x, y) for x, y in zip(*results))


def test_the_calls_are_counted_and_timed():
    b = Batch([1, 200], [50, 260], 4, 2, 128, 32, seed=48)
    k = randn(49, b.cu[-1], 2, 128)
    b.run()
    zl.sync_check()
    zl.profile_begin()
    zl.paged_append_q4(k, k, *b.cache, b.cu)
    zl.paged_read_q4(*b.cache, b.cu)
    b.run()
    names = zl.profile_end()
    assert {"paged_append_q4", "paged_read_q4", "paged_unpack_q4", "paged_attn"} <= set(names)
