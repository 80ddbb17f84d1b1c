"""Whole-page operations on the GPU against a model on Python lists: tables,
lengths and counts equal, and every page of every group where it belongs."""
import numpy as np
import pytest
import torch

import mixed_length_dit_gb300 as zl
from oracle import paged_f64 as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """The device tables beside their model; every page of group g starts as
    page number * 8 + g."""

    def __init__(self, lens, pages, page, cols, spare_slots=0, groups=2, seed=0, elems=(1, 64)):
        rng = np.random.default_rng(seed)
        used = [-(-n // page) for n in lens]
        numbers = rng.permutation(pages)
        table = [[-1] * cols for _ in range(len(lens) + spare_slots)]
        refs, at = [0] * pages, 0
        for s, n in enumerate(used):
            table[s][:n] = [int(x) for x in numbers[at:at + n]]
            for x in table[s][:n]:
                refs[x] = 1
            at += n
        self.m = ref.Pages(table, list(lens) + [0] * spare_slots, refs, page)
        self.table, self.lens, self.refs = i32(table), i32(self.m.lens), i32(refs)
        nk, hd = elems
        self.cache = (torch.arange(pages, device="cuda")[None] * 8 + torch.arange(groups, device="cuda")[:, None])
        self.cache = self.cache.to(torch.int32).view(groups, pages, 1, 1, 1).expand(groups, pages, nk, page, hd // 2)
        self.cache = self.cache.contiguous().view(torch.bfloat16)

    def same(self):
        zl.sync_check()
        assert self.lens.tolist() == self.m.lens
        assert self.refs.tolist() == self.m.refs
        assert self.table.tolist() == self.m.table

    def same_data(self):
        got = self.cache.view(torch.int32)
        for p, d in enumerate(self.m.data):
            if self.m.refs[p] > 0:
                for g in range(got.shape[0]):
                    assert torch.all(got[g, p] == d * 8 + g), (p, g)


@pytest.mark.parametrize("page,pages,slots", [(16, 40, 5), (32, 3000, 60), (256, 20, 8)])
def test_extend(page, pages, slots):
    rng = np.random.default_rng(page)
    b = Both([int(x) for x in rng.integers(0, 3 * page, slots - 1)] + [0], pages, page, 12, seed=page)
    for most in (0, 1, page, 2 * page + 3, 1):
        counts = [int(x) for x in rng.integers(0, most + 1, slots)]
        st = zl.pages_extend(b.table, b.lens, b.refs, i32(counts), page)
        assert int(st) == b.m.extend(counts)
        b.same()


def test_extend_of_many_slots_in_a_large_pool():
    slots, pages, page = 8192, 70000, 16
    rng = np.random.default_rng(8)
    b = Both([int(x) for x in rng.integers(0, 40, slots)], pages, page, 8, seed=8, groups=1)
    counts = [int(x) for x in rng.integers(0, 80, slots)]
    assert int(zl.pages_extend(b.table, b.lens, b.refs, i32(counts), page)) == b.m.extend(counts) == 0
    b.same()
    free = b.m.refs.count(0)
    counts = [16 * (free // slots + 1)] * slots
    assert int(zl.pages_extend(b.table, b.lens, b.refs, i32(counts), page)) == b.m.extend(counts) != 0
    b.same()


def test_extend_that_cannot_be_met_changes_nothing():
    b = Both([20, 5, 0], 6, 16, 4)
    for counts, want in (([44, 20, 16], 1), ([0, -1, 0], -1), ([45, 0, 0], -1), ([2 ** 31 - 1, 0, 0], -1),
                         ([44, 59, 64], 6)):     # 2 + 3 + 4 pages wanted, 3 free
        st = zl.pages_extend(b.table, b.lens, b.refs, i32(counts), 16)
        b.same()
        assert int(st) == want, counts
    assert int(zl.pages_extend(b.table, b.lens, b.refs, i32([44, 4, 16]), 16)) == b.m.extend([44, 4, 16]) == 0
    b.same()


@pytest.mark.parametrize("groups,elems", [(1, (1, 64)), (5, (3, 128)), (16, (8, 128))])
def test_fork(groups, elems):
    b = Both([33, 16, 0, 100, 47], 60, 16, 10, spare_slots=7, groups=groups, elems=elems)
    parents, children = [0, 3, 3, 1, 2, 0], [11, 5, 7, 6, 9, 8]
    st = zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32(parents), i32(children))
    assert int(st) == b.m.fork(parents, children) == 0
    b.same()
    b.same_data()


@pytest.mark.parametrize("parents,children", [
    ([0], [1]), ([0, 0], [4, 4]), ([0], [0]), ([0], [9]), ([-1], [4]), ([5, 0], [4, 99]), ([0, 1, 0], [4, 5, 1]),
])
def test_fork_refused_changes_nothing(parents, children):
    b = Both([33, 16, 8], 12, 16, 6, spare_slots=4)
    st = zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32(parents), i32(children))
    b.same()
    b.same_data()
    assert int(st) == b.m.fork(parents, children) == -1


def test_fork_without_enough_pages():
    b = Both([33, 16, 8], 6, 16, 6, spare_slots=4)          # 5 of 6 pages used... one is free
    st = zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([0, 2, 1]), i32([3, 4, 5]))
    assert int(st) == b.m.fork([0, 2, 1], [3, 4, 5]) == 1
    b.same()
    st = zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([0, 1]), i32([3, 5]))
    assert int(st) == b.m.fork([0, 1], [3, 5]) == 0
    b.same()
    b.same_data()
    empty = i32([])
    assert int(zl.pages_fork(b.cache, b.table, b.lens, b.refs, empty, empty)) == 0
    b.same()


def test_free_shared_and_named_twice():
    b = Both([33, 16, 8], 30, 16, 6, spare_slots=4)
    zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([0, 0]), i32([3, 4]))
    b.m.fork([0, 0], [3, 4])
    zl.pages_free(b.table, b.lens, b.refs, i32([0, 3, 0, 6, 3]), 16)
    b.m.release([0, 3, 0, 6, 3])
    b.same()
    zl.pages_free(b.table, b.lens, b.refs, i32([]), 16)
    b.same()
    zl.pages_free(b.table, b.lens, b.refs, i32([1, 99, -1]), 16)
    b.m.release([1])
    with pytest.raises(zl.ZlError) as e:
        b.same()
    assert e.value.status == -8
    b.same()


@pytest.mark.parametrize("pages,lens,groups,elems", [
    (12, [33, 16, 8], 2, (1, 64)), (500, [1000, 3000, 17, 0, 900], 3, (2, 128)), (4000, [16 * 700] * 3, 2, (1, 64)),
    (5, [80], 1, (1, 64)), (7, [0], 1, (1, 64)),
])
def test_compact(pages, lens, groups, elems):
    b = Both(lens, pages, 16, max(1, max(-(-n // 16) for n in lens)), groups=groups, elems=elems, spare_slots=1)
    live = zl.pages_compact(b.cache, b.table, b.lens, b.refs)
    assert int(live) == b.m.compact()
    b.same()
    b.same_data()
    assert all(r == 0 for r in b.m.refs[int(live):])
    live = zl.pages_compact(b.cache, b.table, b.lens, b.refs)      # nothing left to move
    assert int(live) == b.m.compact()
    b.same()
    b.same_data()


def test_compact_a_large_pool():
    b = Both([16 * 9] * 3000, 60000, 16, 9, seed=9, groups=1)
    rng = np.random.default_rng(9)
    gone = [int(x) for x in rng.permutation(3000)[:1200]]
    zl.pages_free(b.table, b.lens, b.refs, i32(gone), 16)
    b.m.release(gone)
    assert int(zl.pages_compact(b.cache, b.table, b.lens, b.refs)) == b.m.compact()
    b.same()
    got = b.cache.view(torch.int32).view(60000, -1)[:, 0].tolist()
    assert all(got[p] == d * 8 for p, d in enumerate(b.m.data) if b.m.refs[p] > 0)


def test_compact_of_shared_pages():
    b = Both([33, 160, 8], 64, 16, 12, spare_slots=5, seed=3)
    zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([1, 1, 0]), i32([3, 4, 7]))
    b.m.fork([1, 1, 0], [3, 4, 7])
    zl.pages_free(b.table, b.lens, b.refs, i32([1, 2]), 16)
    b.m.release([1, 2])
    assert int(zl.pages_compact(b.cache, b.table, b.lens, b.refs)) == b.m.compact()
    b.same()
    b.same_data()


def test_copy():
    b = Both([160], 40, 16, 12, groups=3, elems=(5, 64))
    before = b.cache.clone()
    src, dst = [3, 3, 20, 39], [0, 7, 8, 9]
    zl.pages_copy(b.cache, i32(src), i32(dst))
    before[:, dst] = before[:, src]
    zl.sync_check()
    assert torch.equal(b.cache.view(torch.int16), before.view(torch.int16))
    zl.pages_copy(b.cache, i32([]), i32([]))
    zl.pages_copy(b.cache, i32([1, 40, -1, 2]), i32([30, 31, 32, 40]))     # pages that are not there
    before[:, 30] = before[:, 1]
    with pytest.raises(zl.ZlError) as e:
        zl.sync_check()
    assert e.value.status == -8
    assert torch.equal(b.cache.view(torch.int16), before.view(torch.int16))


def test_a_captured_loop():
    """Extend, fork and free inside one graph, replayed."""
    b = Both([30, 5], 64, 16, 20, spare_slots=2)
    counts, status = i32([3, 1, 0, 2]), [i32([9]) for _ in range(2)]
    parents, children, slots = i32([0, 1]), i32([2, 3]), i32([3, 2])
    ws = zl.alloc_workspace(zl.pages_workspace_bytes(64), "cuda")
    table0, lens0, refs0 = b.table.clone(), b.lens.clone(), b.refs.clone()

    def once():
        zl.pages_fork(b.cache, b.table, b.lens, b.refs, parents, children, status=status[0], workspace=ws)
        zl.pages_extend(b.table, b.lens, b.refs, counts, 16, status=status[1])
        zl.pages_free(b.table, b.lens, b.refs, slots, 16)
    once()
    b.table.copy_(table0), b.lens.copy_(lens0), b.refs.copy_(refs0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        once()
    for _ in range(7):
        g.replay()
        assert b.m.fork([0, 1], [2, 3]) == int(status[0]) == 0
        assert b.m.extend([3, 1, 0, 2]) == int(status[1]) == 0
        b.m.release([3, 2])
        b.same()


@pytest.mark.parametrize("page,slots", [(16, 5), (32, 300), (256, 8)])
def test_truncate(page, slots):
    rng = np.random.default_rng(page)
    cols = 300 if slots == 5 else 7            # of 300 pages some threads take two
    b = Both([int(x) for x in rng.integers(0, cols * page, slots - 1)] + [0], cols * slots, page, cols)
    for most in (cols * page, cols * page // 2, 2 * page, page, 1, 0):
        keep = [int(x) for x in rng.integers(0, most + 1, slots)]
        zl.pages_truncate(b.table, b.lens, b.refs, i32(keep), page)
        b.m.truncate(keep)
        b.same()
        assert sum(b.m.refs) == sum(b.m.used(n) for n in b.m.lens)   # no page is lost
        counts = [int(x) for x in rng.integers(0, page, slots)]
        assert int(zl.pages_extend(b.table, b.lens, b.refs, i32(counts), page)) == b.m.extend(counts)
        b.same()


def test_truncate_shared_pages_bad_lengths_and_graphs():
    b = Both([70, 16, 8], 30, 16, 6, spare_slots=3)
    zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([0, 0]), i32([3, 4]))
    b.m.fork([0, 0], [3, 4])
    keep = i32([32, 99, 0, 33, 70, 5])
    before = [x.clone() for x in (b.table, b.lens, b.refs)]
    zl.pages_truncate(b.table, b.lens, b.refs, keep, 16)
    b.m.truncate(keep.tolist())
    b.same()
    want = [x.clone() for x in (b.table, b.lens, b.refs)]
    for x, y in zip((b.table, b.lens, b.refs), before):
        x.copy_(y)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        zl.pages_truncate(b.table, b.lens, b.refs, keep, 16)
    for _ in range(2):                         # the second finds nothing left to do
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((b.table, b.lens, b.refs), want))
    # a negative length is flagged, and leaves its slot alone
    zl.pages_truncate(b.table, b.lens, b.refs, i32([-1, 16, 0, 0, 70, 0]), 16)
    b.m.truncate([32, 16, 0, 0, 70, 0])
    with pytest.raises(zl.ZlError) as e:
        b.same()
    assert e.value.status == -8
    b.same()


def test_a_slot_cut_inside_a_shared_page_does_not_grow_over_the_other():
    """Fork, truncate to before the fork, go on: the sibling keeps its tokens,
    and a fork gives the shortened slot a page of its own."""
    b = Both([70, 8], 30, 16, 6, spare_slots=3)
    zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([0]), i32([2]))
    b.m.fork([0], [2])
    keep = [70, 8, 40, 0, 0]                     # slot 2: 8 tokens into a page that slot 0 holds too
    zl.pages_truncate(b.table, b.lens, b.refs, i32(keep), 16)
    b.m.truncate(keep)
    b.same()
    for counts, want in (([0, 0, 1, 0, 0], -2), ([3, 2, 8, 1, 0], -2), ([0, 0, 9, 0, 500], -1), ([1, 1, 0, 1, 1], 0),
                         ([0, 0, 2, 0, 0], -2), ([0, 0, 1, 16 * 90, 0], -1)):
        st = zl.pages_extend(b.table, b.lens, b.refs, i32(counts), 16)
        assert int(st) == b.m.extend(counts) == want, counts
        b.same()
    zl.pages_free(b.table, b.lens, b.refs, i32([3, 4]), 16)
    b.m.release([3, 4])
    assert int(zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([2]), i32([4]))) == b.m.fork([2], [4]) == 0
    zl.pages_free(b.table, b.lens, b.refs, i32([2]), 16)
    b.m.release([2])
    b.same()
    b.same_data()
    assert int(b.table[4, 2]) != int(b.table[0, 2])
    assert int(zl.pages_extend(b.table, b.lens, b.refs, i32([0, 0, 0, 0, 30]), 16)) == b.m.extend([0, 0, 0, 0, 30]) == 0
    b.same()
    b.same_data()
    # a cut at a page's end shares full pages only, and a page whose other holder is gone is one's own again
    zl.pages_fork(b.cache, b.table, b.lens, b.refs, i32([0]), i32([2]))
    b.m.fork([0], [2])
    keep = [71, 9, 32, 0, 70]
    zl.pages_truncate(b.table, b.lens, b.refs, i32(keep), 16)
    b.m.truncate(keep)
    assert int(zl.pages_extend(b.table, b.lens, b.refs, i32([0, 0, 20, 0, 0]), 16)) == b.m.extend([0, 0, 20, 0, 0]) == 0
    b.same()
    zl.pages_truncate(b.table, b.lens, b.refs, i32([71, 9, 25, 0, 70]), 16)
    b.m.truncate([71, 9, 25, 0, 70])
    assert int(zl.pages_extend(b.table, b.lens, b.refs, i32([0, 0, 1, 0, 0]), 16)) == b.m.extend([0, 0, 1, 0, 0]) == -2
    zl.pages_free(b.table, b.lens, b.refs, i32([0, 4]), 16)
    b.m.release([0, 4])
    assert int(zl.pages_extend(b.table, b.lens, b.refs, i32([0, 0, 9, 0, 0]), 16)) == b.m.extend([0, 0, 9, 0, 0]) == 0
    b.same()


def test_tokens_appended_after_a_cut_leave_the_sibling_alone():
    """The loop that a search runs: fork, cut, extend, append.  What the refused
    extend left is what it was, and the sibling's keys stay."""
    page, kv, hd = 16, 2, 64
    cache = torch.zeros((2, 20, kv, page, hd), dtype=torch.bfloat16, device="cuda")
    table, lens, refs = torch.full((2, 6), -1, dtype=torch.int32, device="cuda"), i32([0, 0]), i32([0] * 20)
    plan = zl.RopePlan(hd)
    first = torch.randn((40, kv, hd), device="cuda").to(torch.bfloat16)
    assert int(zl.pages_extend(table, lens, refs, i32([40, 0]), page)) == 0
    zl.paged_append(first, first, *cache, table, lens, [0, 40, 40], rope=plan)
    assert int(zl.pages_fork(cache, table, lens, refs, i32([0]), i32([1]))) == 0
    zl.pages_truncate(table, lens, refs, i32([40, 20]), page)
    before = [x.clone() for x in (cache, table, lens, refs)]
    assert int(zl.pages_extend(table, lens, refs, i32([0, 4]), page)) == -2
    zl.sync_check()
    assert all(torch.equal(x, y) for x, y in zip((cache, table, lens, refs), before))
