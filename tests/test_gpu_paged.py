"""The paged cache's append and attention on the GPU against the float64
definition.

Tolerance of an output element o with reach r = sum_j p_j |v_j| (derived, per
element): each probability is rounded to bf16 once (2^-8 of it at most), so the
sum is off by 2^-8 r; the result is rounded once, 2^-8 |o|; the scores' float32
sums (at most 128 terms of products exact in float32, truncated at worst:
128 * 2^-23 * sum|q_i k_i| * scale, under 2e-4 for the inputs here) and the
exponential (2^-22) move every probability by under 2^-11 of it, numerator and
denominator both.  LSE: the scores' 2e-4, and 2^-20 of its value.
"""
import numpy as np
import pytest
import torch

import mixed_length_dit_gb300 as zl
from oracle import paged_f64 as ref
from _helpers import f64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class Batch:
    """New tokens and a cache in use: pages in any order, pool rows and table
    entries that belong to nobody filled with what must not matter."""

    def __init__(self, new, lens, heads, kv_heads, hd, page, seed=0, spare_cols=2, fill=float("nan")):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.lens, self.hd, self.page = list(new), list(lens), hd, page
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
        shape = (self.num_pages, kv_heads, page, hd)
        self.k_pages, self.v_pages = (torch.randn(shape, generator=g, device="cuda").to(BF16) for _ in range(2))
        for s, n in enumerate(lens):
            if n % page:
                for p in (self.k_pages, self.v_pages):
                    p[int(self.table[s, n // page]), :, n % page:] = fill
        for p in numbers[at:]:
            self.k_pages[int(p)] = fill
            self.v_pages[int(p)] = fill
        self.q = torch.randn((self.cu[-1], heads, hd), generator=g, device="cuda").to(BF16)
        self.dtable = torch.tensor(self.table, device="cuda")
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def run(self, q=None, most=None, **kw):
        q = self.q if q is None else q
        return zl.paged_attn(q, self.k_pages, self.v_pages, self.dtable, self.dlens, self.cu,
                             max(self.lens) if most is None else most, **kw)

    def check(self, o, lse, **kw):
        want, want_lse, reach = ref.paged_attn(f64(self.q), f64(self.k_pages), f64(self.v_pages), self.table, self.lens,
                                               self.cu, **kw)
        tol = (2.0 ** -8 + 2.0 ** -11) * reach + 2.0 ** -8 * np.abs(want)
        err = np.abs(f64(o) - want)
        assert np.all(err <= tol), float((err - tol).max())
        none = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(f64(lse)), none)
        fin = ~none
        err = np.abs(f64(lse)[fin] - want_lse[fin])
        assert np.all(err <= 2e-4 + 2.0 ** -20 * np.abs(want_lse[fin])), float(err.max())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 1), (10, 2), (6, 2), (40, 8)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(heads, kv_heads, hd, page):
    b = Batch([1] * 6, [1, 2, 127, 128, 129, 700], heads, kv_heads, hd, page)
    o, lse = b.run()
    zl.sync_check()
    b.check(o, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,kv_heads,hd,page", [(2, 2, 64, 16), (6, 2, 128, 32), (10, 2, 128, 128), (7, 1, 64, 64)])
def test_chunks(heads, kv_heads, hd, page, causal):
    new = [130, 1, 300, 0, 37, 128, 2, 257]
    lens = [130, 500, 431, 90, 300, 1000, 64, 258]
    b = Batch(new, lens, heads, kv_heads, hd, page, seed=1)
    o, lse = b.run(causal=causal)
    zl.sync_check()
    b.check(o, lse, causal=causal)


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 7), (True, 128), (True, 200), (False, 33), (False, 129),
                                           (True, 10 ** 6)])
def test_windows(causal, window):
    b = Batch([1, 260, 33, 5], [900, 500, 33, 389], 6, 2, 64, 32, seed=2)
    o, lse = b.run(causal=causal, window=window)
    zl.sync_check()
    b.check(o, lse, causal=causal, window=window)


@pytest.mark.parametrize("group", [3, 5, 7, 12, 48, 100, 128])
def test_many_heads_of_one_key_head(group):
    b = Batch([1, 9, 40], [300, 140, 44], group, 1, 64, 16, seed=3)
    o, lse = b.run()
    zl.sync_check()
    b.check(o, lse)


def test_long_cache_is_split_and_joined():
    b = Batch([1, 3, 1], [20011, 513, 6000], 8, 2, 128, 64, seed=4)
    for kw in ({}, {"window": 4097}, {"causal": False}):
        o, lse = b.run(**kw)
        zl.sync_check()
        b.check(o, lse, **kw)
    # a larger bound of the lengths changes the split, not the result
    o, lse = b.run(most=b.dtable.shape[1] * b.page)
    b.check(o, lse)


def test_a_serving_batch_of_long_ragged_sequences():
    """More work items than SMs, each of many key blocks, taken over and over:
    sampled rows against the definition in 64 bits, and the same bits again."""
    lens = [1501 + i * 12701 % 14885 for i in range(48)]
    b = Batch([1] * 48, lens, 40, 8, 128, 16, seed=16, fill=1.0)
    o, lse = b.run()
    for _ in range(20):
        o2, l2 = b.run()
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    zl.sync_check()
    for s in range(0, 48, 5):
        rows = b.dtable[s, :-(-lens[s] // 16)].long()
        k, v = (x[rows].transpose(1, 2).flatten(0, 1)[:lens[s]].double() for x in (b.k_pages, b.v_pages))
        for h in range(0, 40, 3):
            p = (k[:, h // 5] @ b.q[s, h].double()) * 128 ** -0.5
            w = torch.softmax(p, 0)
            want, reach = w @ v[:, h // 5], w @ v[:, h // 5].abs()
            assert torch.all((o[s, h].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * reach + 2.0 ** -8 * want.abs())
            assert abs(float(lse[h, s].double() - torch.logsumexp(p, 0))) <= 2e-4 + 2.0 ** -20 * 15


def test_few_chunk_rows_over_a_long_cache():
    b = Batch([140, 5], [9000, 333], 2, 1, 64, 16, seed=5)
    for kw in ({}, {"causal": False}, {"window": 2500}):
        o, lse = b.run(**kw)
        zl.sync_check()
        b.check(o, lse, **kw)


def test_rows_that_see_nothing():
    """Lengths shorter than the chunk (positions below zero) and empty ones."""
    b = Batch([5, 3, 1, 200], [2, 0, 0, 150], 4, 2, 64, 16, seed=6)
    for kw in ({}, {"causal": False}, {"window": 2}):
        o, lse = b.run(**kw)
        zl.sync_check()
        b.check(o, lse, **kw)
        assert torch.isfinite(o.float()).all()
    assert torch.all(o[5:9] == 0)


@pytest.mark.parametrize("fill", [float("inf"), float("-inf"), 3e38])
def test_what_belongs_to_nobody_does_not_matter(fill):
    b = Batch([1, 40], [77, 100], 4, 2, 128, 64, seed=7, fill=fill)
    o, lse = b.run()
    zl.sync_check()
    b.check(o, lse)


def test_non_finite_keys_past_the_mask():
    """A key that a query does not see may hold anything."""
    b = Batch([60], [300], 4, 2, 64, 16, seed=8)
    last = f64(b.k_pages)
    o1, l1 = b.run()
    b.k_pages[int(b.table[0, 299 // 16]), :, 299 % 16] = float("nan")    # the newest token's key
    o2, l2 = b.run()
    zl.sync_check()
    assert torch.equal(o1[:59], o2[:59]) and torch.equal(l1[:, :59], l2[:, :59])
    assert np.isfinite(last[int(b.table[0, 0])]).all()


def test_large_scores():
    """Scores of thousands, whose running maximum jumps block by block."""
    b = Batch([1, 50], [700, 700], 4, 2, 64, 16, seed=9)
    b.q *= 64
    o, lse = b.run(softmax_scale=1.0)
    zl.sync_check()
    want, want_lse, _ = ref.paged_attn(f64(b.q), f64(b.k_pages), f64(b.v_pages), b.table, b.lens, b.cu, scale=1.0)
    # scores reach 64 * 64 * 4: their sums' 64 * 2^-23 * sum|q k| (about 3,300) is 0.03 of a logit
    assert np.abs(f64(lse) - want_lse).max() <= 0.03 + 2.0 ** -20 * np.abs(want_lse).max()
    assert np.abs(f64(o) - want).max() <= 0.07 * np.abs(f64(b.v_pages)[b.table[0, :43]]).max() + 2.0 ** -7 * np.abs(want).max()


def test_queries_inside_wider_rows_and_given_buffers():
    b = Batch([1, 200, 7], [50, 260, 130], 6, 2, 128, 32, seed=10)
    o1, l1 = b.run()
    rows = torch.randn((b.cu[-1], 10, 128), device="cuda").to(BF16)
    rows[:, 2:8] = b.q
    out = torch.full_like(o1, 9.0)
    lse = torch.full_like(l1, 9.0)
    ws = zl.alloc_workspace(zl.paged_attn_workspace_bytes(b.cu, max(b.lens), 6, 2, 128), "cuda")
    o2, l2 = b.run(q=rows[:, 2:8], out=out, lse=lse, workspace=ws)
    assert o2 is out and l2 is lse and torch.equal(o1, out) and torch.equal(l1, lse)


def test_small_workspace_is_refused():
    b = Batch([1], [20000], 2, 1, 64, 64, seed=11)
    need = zl.paged_attn_workspace_bytes(b.cu, 20000, 2, 1, 64)
    if need == 0:
        pytest.skip("nothing is split here")
    with pytest.raises(zl.ZlError) as e:
        b.run(workspace=torch.empty(need - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4


def test_more_sequences_than_one_launch_holds():
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(1, 90, 700)]
    b = Batch([1] * 700, lens, 2, 1, 64, 16, seed=12)
    o, lse = b.run()
    zl.sync_check()
    b.check(o, lse)


def test_same_bits_every_time():
    b = Batch([1, 300, 2], [5000, 900, 2500], 8, 2, 128, 16, seed=13)
    o, lse = b.run()
    for _ in range(3):
        o2, l2 = b.run()
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_pages_and_lengths_out_of_range_are_left_out_and_reported():
    b = Batch([1, 1, 4], [100, 90, 60], 4, 2, 64, 16, seed=14)
    b.dtable[1, 2] = b.num_pages
    b.run()
    with pytest.raises(zl.ZlError) as e:
        zl.sync_check()
    assert e.value.status == -8
    b.dtable[1, 2] = -7
    o, lse = b.run()
    with pytest.raises(zl.ZlError):
        zl.sync_check()
    b.dtable[1, 2] = int(b.table[1, 2])
    b.dlens[1] = 5000                     # past the bound that was given
    o, lse = b.run()
    with pytest.raises(zl.ZlError):
        zl.sync_check()
    b.dlens[1] = -3
    o, lse = b.run()
    with pytest.raises(zl.ZlError):
        zl.sync_check()
    b.dlens[1] = 90
    o, lse = b.run()
    zl.sync_check()
    b.check(o, lse)


def test_graph_replays_with_the_lengths_and_pages_of_the_moment():
    b = Batch([1, 1, 1], [40, 2500, 333], 8, 2, 128, 16, seed=15, spare_cols=6)
    most = b.dtable.shape[1] * 16
    out, lse = torch.zeros_like(b.q), torch.zeros((8, 3), device="cuda")
    ws = zl.alloc_workspace(zl.paged_attn_workspace_bytes(b.cu, most, 8, 2, 128), "cuda")
    b.run(most=most, out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(most=most, out=out, lse=lse, workspace=ws)
    for lens in ([40, 2500, 333], [33, 17, 330], [1, 1290, 16]):
        b.lens = lens
        b.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        zl.sync_check()
        b.check(out, lse)


def test_two_streams_at_once():
    bs = [Batch([1, 90], [3000 + 500 * i, 300], 8, 2, 128, 16, seed=20 + i) for i in range(2)]
    want = [b.run() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    got = []
    for _ in range(5):
        for b, s in zip(bs, streams):
            got.append(b.run(stream=s))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_two_graphs_share_a_workspace():
    bs = [Batch([1, 3], [3000, 700], 8, 2, 128, 16, seed=50), Batch([200, 1], [900, 2000], 8, 2, 128, 16, seed=51)]
    want = [b.run() for b in bs]
    size = max(zl.paged_attn_workspace_bytes(b.cu, max(b.lens), 8, 2, 128) for b in bs)
    ws = zl.alloc_workspace(size, "cuda")
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


def test_no_key_at_all():
    b = Batch([2, 200], [16, 16], 4, 2, 64, 16, seed=52)
    b.dlens.zero_()
    for most in (0, 16):
        o, lse = b.run(most=most)
        zl.sync_check()
        assert torch.all(o == 0) and torch.isneginf(lse).all()


@pytest.mark.parametrize("new", [1, 20])
def test_windows_as_large_as_an_int(new):
    """A window over everything is no window, also for positions below zero."""
    b = Batch([new, new], [10, 300], 4, 1, 64, 16, seed=53)
    for causal in (True, False):
        want = b.run(causal=causal)
        got = b.run(causal=causal, window=2 ** 31 - 1)
        zl.sync_check()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        b.check(*got, causal=causal)


def test_offsets_past_32_bits():
    """Pools of more than 2^31 elements, of which the last pages are used: the
    same bits as with a small pool."""
    small = Batch([1, 150, 4], [700, 400, 4], 8, 8, 128, 128, seed=54, fill=1.0)
    k, v = (torch.randn((155, 8, 128), device="cuda").to(BF16) for _ in range(2))
    plan = zl.RopePlan(128)
    pages = 2 ** 31 // (8 * 128 * 128) + 40
    big = [torch.empty((pages, 8, 128, 128), dtype=BF16, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 31
    shift = pages - small.num_pages
    for x, y in zip(big, (small.k_pages, small.v_pages)):
        x[shift:] = y
    used = (torch.arange(small.dtable.shape[1], device="cuda") < (small.dlens[:, None] + 127) // 128)
    table = torch.where(used, small.dtable + shift, -1).int()
    q1 = zl.paged_append(k, v, small.k_pages, small.v_pages, small.dtable, small.dlens, small.cu, q=small.q, rope=plan)
    q2 = zl.paged_append(k, v, *big, table, small.dlens, small.cu, q=small.q, rope=plan)
    zl.sync_check()
    assert torch.equal(q1, q2) and torch.equal(big[0][shift:], small.k_pages) and torch.equal(big[1][shift:], small.v_pages)
    o1, l1 = zl.paged_attn(q1, small.k_pages, small.v_pages, small.dtable, small.dlens, small.cu, 700)
    o2, l2 = zl.paged_attn(q1, *big, table, small.dlens, small.cu, 700)
    zl.sync_check()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    last = torch.tensor([pages - 1], dtype=torch.int32, device="cuda")
    zl.pages_copy(big[0], last, torch.zeros_like(last))
    assert torch.equal(big[0][0], big[0][-1])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("hd,heads,kv_heads,page,axes,il", [
    (64, 4, 2, 16, (64,), False), (128, 10, 2, 64, (128,), True), (128, 3, 3, 256, (64,), False), (64, 2, 1, 32, (6,), True),
])
def test_append_turns_and_writes(hd, heads, kv_heads, page, axes, il):
    new, lens = [1, 40, 0, 200, 3], [90, 40, 5, 333, 259]
    b = Batch(new, lens, heads, kv_heads, hd, page, seed=30, fill=5.0)
    g = torch.Generator(device="cuda").manual_seed(31)
    rows = torch.randn((b.cu[-1], kv_heads * 2, hd), generator=g, device="cuda").to(BF16)
    k, v = rows[:, :kv_heads], rows[:, kv_heads:]
    plan = zl.RopePlan(hd, axes=axes, interleaved=il)
    k0, v0 = f64(b.k_pages), f64(b.v_pages)
    q = zl.paged_append(k, v, b.k_pages, b.v_pages, b.dtable, b.dlens, b.cu, q=b.q, rope=plan)
    zl.sync_check()
    pos = np.concatenate([np.arange(n - m, n) for m, n in zip(new, lens)])[None]
    turned = ref.rope(f64(k), pos, axes, interleaved=il)
    want_v = ref.append(v0, b.table, lens, b.cu, f64(v))
    assert np.array_equal(f64(b.v_pages), want_v)
    want_k = ref.append(k0, b.table, lens, b.cu, turned)
    tol = 2.0 ** -8 * np.abs(want_k) + 2.0 ** -21 * ref.append(0 * k0, b.table, lens, b.cu, ref.rope_reach(f64(k), axes, il))
    tol[want_k == k0] = 0
    assert np.all(np.abs(f64(b.k_pages) - want_k) <= tol)
    want_q = ref.rope(f64(b.q), pos, axes, interleaved=il)
    tol = 2.0 ** -8 * np.abs(want_q) + 2.0 ** -21 * ref.rope_reach(f64(b.q), axes, il)
    assert np.all(np.abs(f64(q) - want_q) <= tol)


def test_append_without_rope_and_with_positions():
    b = Batch([5, 1], [20, 300], 2, 2, 64, 16, seed=32, fill=1.0)
    k, v = torch.randn((6, 2, 64), device="cuda").to(BF16), torch.randn((6, 2, 64), device="cuda").to(BF16)
    k0, v0 = f64(b.k_pages), f64(b.v_pages)
    assert zl.paged_append(k, v, b.k_pages, b.v_pages, b.dtable, b.dlens, b.cu) is None
    assert np.array_equal(f64(b.k_pages), ref.append(k0, b.table, b.lens, b.cu, f64(k)))
    assert np.array_equal(f64(b.v_pages), ref.append(v0, b.table, b.lens, b.cu, f64(v)))
    plan = zl.RopePlan(64, axes=(32, 32))
    pos = torch.tensor([[1, 2, 3, 4, 5, 6], [9, 9, 9, 9, 9, -9]], dtype=torch.int32, device="cuda")
    q = zl.paged_append(k, v, b.k_pages, b.v_pages, b.dtable, b.dlens, b.cu, q=b.q, rope=plan, positions=pos)
    want, _ = zl.rope_fwd(b.q, None, pos, plan)
    assert torch.equal(q, want)
    want, _ = zl.rope_fwd(k, None, pos, plan)
    assert np.array_equal(f64(b.k_pages), ref.append(k0, b.table, b.lens, b.cu, f64(want)))


def test_append_past_the_cache_is_left_out_and_reported():
    b = Batch([3, 2], [30, 20], 2, 1, 64, 16, seed=33, fill=1.0)
    k = torch.randn((5, 1, 64), device="cuda").to(BF16)
    k0 = f64(b.k_pages)
    b.dlens[0] = 10 ** 6                   # far past the table row
    b.dtable[1, 1] = -1
    zl.paged_append(k, k, b.k_pages, b.v_pages, b.dtable, b.dlens, b.cu)
    with pytest.raises(zl.ZlError) as e:
        zl.sync_check()
    assert e.value.status == -8
    assert np.array_equal(f64(b.k_pages), k0)
    b.dlens[0] = 1                         # shorter than the new tokens: the last of them is its only one
    b.dtable[1, 1] = int(b.table[1, 1])
    zl.paged_append(k, k, b.k_pages, b.v_pages, b.dtable, b.dlens, b.cu)
    with pytest.raises(zl.ZlError):
        zl.sync_check()
    assert np.array_equal(f64(b.k_pages)[b.table[0, 0], 0, 0], f64(k)[2, 0])


def test_append_many_sequences():
    rng = np.random.default_rng(34)
    lens = [int(x) for x in rng.integers(1, 60, 1300)]
    new = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 4, 1300))]
    b = Batch(new, lens, 1, 1, 64, 16, seed=34, fill=1.0)
    k = torch.randn((b.cu[-1], 1, 64), device="cuda").to(BF16)
    k0 = f64(b.k_pages)
    zl.paged_append(k, k, b.k_pages, b.v_pages, b.dtable, b.dlens, b.cu)
    zl.sync_check()
    assert np.array_equal(f64(b.k_pages), ref.append(k0, b.table, b.lens, b.cu, f64(k)))


# ------------------------------------------------------------------ a run of them together
def test_generation_loop():
    """Prompts, single tokens, a fork, more tokens, a sequence freed and the
    pool compacted, on one cache of two layers; every step's attention equals
    the packed attention over the sequences' whole histories."""
    layers, page, hd, heads, kv, slots, pages = 2, 16, 64, 4, 2, 6, 60
    g = torch.Generator(device="cuda").manual_seed(40)
    cache = torch.full((layers, 2, pages, kv, page, hd), float("nan"), dtype=BF16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.full((slots, 12), -1, dtype=torch.int32, device="cuda")
    lens, refs = i32([0] * slots), i32([0] * pages)
    plan = zl.RopePlan(hd)
    past = [[] for _ in range(slots)]          # per slot and layer: (k, v) rows as appended, unturned
    past = [[[] for _ in range(layers)] for _ in range(slots)]
    host = ref.Pages(table.tolist(), [0] * slots, [0] * pages, page)

    def step(counts):
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        status = zl.pages_extend(table, lens, refs, i32(counts), page)
        assert host.extend(counts) == int(status) == 0
        for layer in range(layers):
            q = torch.randn((cu[-1], heads, hd), generator=g, device="cuda").to(BF16)
            k, v = (torch.randn((cu[-1], kv, hd), generator=g, device="cuda").to(BF16) for _ in range(2))
            kp, vp = cache[layer]
            qr = zl.paged_append(k, v, kp, vp, table, lens, cu, q=q, rope=plan)
            o, lse = zl.paged_attn(qr, kp, vp, table, lens, cu, 12 * page)
            zl.sync_check()
            for s in range(slots):
                if counts[s] == 0:
                    continue
                past[s][layer].append((k[cu[s]:cu[s + 1]], v[cu[s]:cu[s + 1]]))
                kk, vv = (torch.cat([x[i] for x in past[s][layer]]) for i in range(2))
                assert kk.shape[0] == host.lens[s]
                pos = torch.arange(kk.shape[0], dtype=torch.int32, device="cuda")
                kr, _ = zl.rope_fwd(kk, None, pos, plan)
                p0 = kk.shape[0] - counts[s]
                for h in range(heads):
                    want, wl, reach = ref.attn_rows(f64(qr)[cu[s]:cu[s + 1], h], f64(kr)[:, h // 2], f64(vv)[:, h // 2],
                                                    p0 + np.arange(counts[s]), True, 0, hd ** -0.5)
                    err = np.abs(f64(o)[cu[s]:cu[s + 1], h] - want)
                    assert np.all(err <= (2.0 ** -8 + 2.0 ** -11) * reach + 2.0 ** -8 * np.abs(want))
                    assert np.all(np.abs(f64(lse)[h, cu[s]:cu[s + 1]] - wl) <= 2e-4 + 2.0 ** -20 * np.abs(wl))

    step([35, 100, 16, 0, 0, 0])
    step([1, 1, 1, 0, 0, 0])
    assert int(zl.pages_fork(cache, table, lens, refs, i32([1, 1, 2]), i32([3, 5, 4]))) == host.fork([1, 1, 2], [3, 5, 4]) == 0
    for p, c in ((1, 3), (1, 5), (2, 4)):
        past[c] = [list(x) for x in past[p]]
    step([1, 1, 1, 1, 1, 1])
    step([0, 20, 0, 3, 0, 1])
    zl.pages_free(table, lens, refs, i32([0, 5]), page)
    host.release([0, 5])
    past[0], past[5] = ([[] for _ in range(layers)] for _ in range(2))
    assert int(zl.pages_compact(cache, table, lens, refs)) == host.compact()
    assert refs.tolist() == host.refs and lens.tolist() == host.lens
    for s in range(slots):
        assert table[s, :host.used(host.lens[s])].tolist() == host.table[s][:host.used(host.lens[s])]
    step([17, 1, 1, 1, 1, 40])


def test_drafts_taken_back_leave_what_was_never_drafted():
    """Drafted tokens appended, attended to, and in part taken back: the cache
    goes on as if only the accepted ones had been there, bit for bit."""
    page, hd, heads, kv, slots, pages = 16, 128, 8, 2, 3, 40
    g = torch.Generator(device="cuda").manual_seed(41)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    plan = zl.RopePlan(hd)
    rand = lambda n, h: torch.randn((n, h, hd), generator=g, device="cuda").to(BF16)

    class Cache:
        def __init__(self):
            self.kv = torch.zeros((2, pages, kv, page, hd), dtype=BF16, device="cuda")
            self.table = torch.full((slots, 12), -1, dtype=torch.int32, device="cuda")
            self.lens, self.refs = i32([0] * slots), i32([0] * pages)

        def step(self, q, k, v, cu):
            counts = [b - a for a, b in zip(cu, cu[1:])]
            assert int(zl.pages_extend(self.table, self.lens, self.refs, i32(counts), page)) == 0
            qr = zl.paged_append(k, v, self.kv[0], self.kv[1], self.table, self.lens, cu, q=q, rope=plan)
            return zl.paged_attn(qr, self.kv[0], self.kv[1], self.table, self.lens, cu, 12 * page)

    drafted, plain = Cache(), Cache()
    start = [30, 16, 47]
    cu = [0, 30, 46, 93]
    first = rand(93, heads), rand(93, kv), rand(93, kv)
    for c in (drafted, plain):
        c.step(*first, cu)
    for accepted in ([0, 1, 4], [5, 0, 2], [1, 1, 1]):
        q, k, v = rand(15, heads), rand(15, kv), rand(15, kv)
        drafted.step(q, k, v, [0, 5, 10, 15])
        start = [n + a for n, a in zip(start, accepted)]
        zl.pages_truncate(drafted.table, drafted.lens, drafted.refs, i32(start), page)
        rows = [5 * s + i for s in range(slots) for i in range(accepted[s])]
        cu = [0]
        for a in accepted:
            cu.append(cu[-1] + a)
        plain.step(q[rows], k[rows], v[rows], cu)
        assert drafted.lens.tolist() == plain.lens.tolist() == start
        assert int(drafted.refs.sum()) == int(plain.refs.sum())
        q, k, v = rand(slots, heads), rand(slots, kv), rand(slots, kv)
        o, o2 = (c.step(q, k, v, [0, 1, 2, 3]) for c in (drafted, plain))
        zl.sync_check()
        start = [n + 1 for n in start]
        assert torch.equal(o[0], o2[0]) and torch.equal(o[1], o2[1])


@pytest.mark.parametrize("new,lens,heads,kv_heads,hd", [
    ([1, 1], [40, 300], 8, 2, 128), ([12, 3], [200, 90], 10, 2, 64), ([100], [260], 1, 1, 128), ([300, 70], [300, 900], 4, 2, 64),
    ([1], [20000], 6, 2, 128), ([150], [9000], 2, 1, 64),
])
def test_nan_is_handed_on(new, lens, heads, kv_heads, hd):
    """A query or a visible key of NaN makes its rows NaN, as the formula does,
    and no other row's bits change."""
    b = Batch(new, lens, heads, kv_heads, hd, 16, seed=11)
    o1, l1 = b.run()
    q = b.q.clone()
    rows = [0, b.cu[-1] - 1]
    q[rows, heads - 1, 3] = float("nan")
    o2, l2 = b.run(q=q)
    nan = torch.zeros((b.cu[-1], heads), dtype=torch.bool, device="cuda")
    nan[rows, heads - 1] = True
    for hit, o, lse in ((nan, o2, l2),):
        assert o[hit].isnan().all() and lse.T[hit].isnan().all()
        assert torch.equal(o[~hit], o1[~hit]) and torch.equal(lse.T[~hit], l1.T[~hit])
    # the last sequence's newest key: its last query alone sees it
    s, n = len(lens) - 1, lens[-1]
    b.k_pages[int(b.table[s, (n - 1) // 16]), 0, (n - 1) % 16, 0] = float("nan")
    o3, l3 = b.run()
    zl.sync_check()
    nan[:] = False
    nan[-1, :heads // kv_heads] = True
    assert o3[nan].isnan().all() and l3.T[nan].isnan().all()
    assert torch.equal(o3[~nan], o1[~nan]) and torch.equal(l3.T[~nan], l1.T[~nan])


@pytest.mark.parametrize("new,lens,heads,kv_heads,hd", [
    ([1], [700], 8, 8, 64), ([1] * 19, [130] * 18 + [1000], 16, 8, 128), ([3, 1, 2], [3, 0, 600], 12, 4, 64),
    ([200], [600], 4, 4, 128), ([600, 129, 300], [620, 129, 1], 3, 1, 64), ([90, 1, 400, 2], [90, 500, 700, 7], 20, 4, 128),
    ([130] * 5, [0, 1, 200, 640, 64], 6, 2, 64),
])
def test_whole_and_cut_units_agree(new, lens, heads, kv_heads, hd):
    """A bound of the lengths decides whether units are left whole; either way
    the result is the formula's, and the order of units does not matter."""
    b = Batch(new, lens, heads, kv_heads, hd, 32, seed=12, spare_cols=2000)
    for kw in ({}, {"causal": False}, {"window": 100}):
        for most in (max(lens), 60000):
            before = zl.launch_count()
            o, lse = b.run(most=most, **kw)
            launches = zl.launch_count() - before
            zl.sync_check()
            b.check(o, lse, **kw)
            kinds = len({n * (heads // kv_heads) > 128 // (heads // kv_heads) * (heads // kv_heads) for n in new})
            if most == 60000 and "window" not in kw:
                assert launches == 2 * kinds
            else:
                assert kinds <= launches <= 2 * kinds


@pytest.mark.parametrize("hd", [64, 128])
def test_many_rows_of_many_parts(hd):
    """Chunks and drafts of many rows, each row's keys spread over many SMs."""
    for new, lens, heads, kv in (([250], [9000], 1, 1), ([64], [20000], 1, 1), ([30, 25], [15000, 40], 3, 1)):
        b = Batch(new, lens, heads, kv, hd, 64, seed=13)
        o, lse = b.run()
        zl.sync_check()
        b.check(o, lse)


# ------------------------------------------------------------------ an append behind a refused extend
def _small_cache(slots, pages, page=16, kv=2, hd=64):
    cache = torch.zeros((2, pages, kv, page, hd), dtype=BF16, device="cuda")
    table = torch.full((slots, 8), -1, dtype=torch.int32, device="cuda")
    return cache, table, *(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (slots, pages))


@pytest.mark.parametrize("way", ["short", "stream", "positions", "q_out"])
def test_append_behind_a_refused_extend_writes_nothing(way):
    """The lengths are the old ones then: without the status the new tokens
    would replace the last ones, also in pages that a fork shares."""
    page, kv, hd = 16, 2, 64
    cache, table, lens, refs = _small_cache(3, 4)
    plan = zl.RopePlan(hd)
    g = torch.Generator(device="cuda").manual_seed(60)
    rand = lambda n, h: torch.randn((n, h, hd), generator=g, device="cuda").to(BF16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kw = {}
    if way == "stream":
        kw["stream"] = torch.cuda.Stream()
    elif way == "positions":
        kw["positions"] = i32(list(range(22)))

    def append(n, cu, status):
        k, v, q = rand(n, kv), rand(n, kv), rand(n, 4)
        if way == "positions":
            kw["positions"] = i32(list(range(n)))
        if way == "q_out":
            kw["q_out"] = torch.empty_like(q)
        torch.cuda.synchronize()
        zl.paged_append(k, v, *cache, table, lens, cu, q=q, rope=plan, status=status, **kw)
        torch.cuda.synchronize()

    status = zl.pages_extend(table, lens, refs, i32([32, 16, 0]), page)
    assert int(status) == 0
    append(48, [0, 32, 48, 48], status)
    zl.sync_check()
    assert cache[:, :3].float().abs().sum((2, 3, 4)).min() > 0
    assert int(zl.pages_fork(cache, table, lens, refs, i32([0]), i32([2]))) == 0     # full pages, shared
    before = [x.clone() for x in (cache, table, lens, refs)]
    status = zl.pages_extend(table, lens, refs, i32([1, 1, 20]), page)
    assert int(status) == 3
    append(22, [0, 1, 2, 22], status)
    with pytest.raises(zl.ZlError) as e:
        zl.sync_check()
    assert e.value.status == -8
    assert all(torch.equal(x, y) for x, y in zip((cache, table, lens, refs), before))
    status = zl.pages_extend(table, lens, refs, i32([1, 0, 0]), page)                # one page is left
    assert int(status) == 0
    append(1, [0, 1, 1, 1], status)
    zl.sync_check()
    changed = (cache != before[0]).flatten(2).any(2).any(0).tolist()
    assert changed == [p == int(table[0, 2]) for p in range(4)]


def test_a_replayed_loop_that_runs_out_of_pages():
    """Extend and append in one graph: once the pool is full every replay leaves
    the cache as it was, and reports it."""
    page, kv, hd, slots = 16, 2, 64, 700                 # two launches an append
    cache, table, lens, refs = _small_cache(slots, 2 * slots)
    g = torch.Generator(device="cuda").manual_seed(61)
    k, v = (torch.randn((slots * 11, kv, hd), generator=g, device="cuda").to(BF16) for _ in range(2))
    counts = torch.full((slots,), 11, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = zl.host_int32([11 * i for i in range(slots + 1)])

    def once():
        zl.pages_extend(table, lens, refs, counts, page, status=status)
        zl.paged_append(k, v, *cache, table, lens, cu, status=status)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        once()
    for n in (11, 22):
        k.add_(1)
        graph.replay()
        zl.sync_check()
        assert int(status) == 0 and lens.tolist() == [n] * slots
        last = table[:, (n - 1) // page].long()
        assert torch.equal(cache[0][last, :, (n - 1) % page], k[10::11])
    before = [x.clone() for x in (cache, table, lens, refs)]
    for _ in range(2):                                   # 33 tokens take three pages a slot
        k.add_(1)
        graph.replay()
        with pytest.raises(zl.ZlError):
            zl.sync_check()
        assert int(status) == slots
        assert all(torch.equal(x, y) for x, y in zip((cache, table, lens, refs), before))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,new,lens,kw", [
    (40, 40, [512, 512], [90, 40], {}),               # of each pair of tiles that sees a key, the first sees none
    (48, 16, [200, 160, 85], [60, 20, 1], {}),        # three heads to a row's token: tiles of 42
    (32, 32, [512] * 3, [300, 100, 512], {"window": 5}),
    (64, 64, [256] * 3, [100, 120, 90], {"window": 3}),
])
def test_items_whose_tiles_see_nothing_in_turn(heads, kv_heads, new, lens, kw, hd):
    """Lengths shorter than the chunk, of many key heads: a CTA meets one item
    after the other in which one of its two tiles has no key block."""
    b = Batch(new, lens, heads, kv_heads, hd, 16, seed=62, spare_cols=2000)
    o, lse = b.run(most=30000, **kw)
    zl.sync_check()
    b.check(o, lse, **kw)
    for _ in range(30):
        o2, l2 = b.run(most=30000, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    zl.sync_check()


@pytest.mark.parametrize("slots", [70, 700])
def test_more_chunks_than_few_and_than_one_launch_holds(slots):
    rng = np.random.default_rng(63)
    new = [int(x) for x in rng.choice([0, 1, 129, 140], slots)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 60, slots))]
    b = Batch(new, lens, 1, 1, 64, 16, seed=63)
    o, lse = b.run()
    zl.sync_check()
    b.check(o, lse)
