"""The device status behind calls of branching requests: an error exactly where
a reference finds something unsound, from captured calls and from two streams."""
import random

import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import check, pages_of
from _pages import bits, compact_reference, copy_reference, fork_reference, free_reference
from _tree import TreeProblem, random_tree

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
PS, PAGES, WIDTH, ROWS = 16, 160, 6, 10


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _status():
    torch.cuda.synchronize()
    return _lib.fa_get_device_status()


class Step:
    """Forks, copies, moves and ends of one pool, in buffers that stay."""

    def __init__(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.r = random.Random(seed)
        self.caches = [torch.randint(-32768, 32768, (PAGES, 2, PS, 64), generator=g, device="cuda",
                                     dtype=torch.int16).view(BF) for _ in range(2)]
        self.src, self.dst, self.lens, self.table = _i32([0] * 4), _i32([0] * 4), _i32([0] * ROWS), _i32([[0] * WIDTH] * ROWS)
        self.free, self.start, self.shares = _i32([0] * 40), _i32([0]), _i32([0] * PAGES)
        self.keep, self.keep_lens, self.base, self.ends = _i32([[0] * 8] * ROWS), _i32([0] * ROWS), _i32([0] * ROWS), _i32([0] * ROWS)

    def fill(self, start, fault=None):
        """A step of six requests, four of which branch; returns whether it is sound."""
        r = self.r
        n = [r.randint(17, PS * WIDTH) for _ in range(6)] + [0] * 4
        ids = r.sample(range(PAGES), PAGES)
        table = [[ids.pop() for _ in range(WIDTH)] for _ in range(6)] + [[-1] * WIDTH for _ in range(4)]
        pool, zero = ids[:40], [0] * PAGES
        src, dst = [r.randrange(3) for _ in range(4)], [6, 7, 8, 9]
        keep = [sorted(r.sample(range(n[b]), min(8, n[b] // 2))) if 3 <= b < 6 else [] for b in range(ROWS)]
        if fault == "length":
            n[src[0]] = PS * WIDTH + 1
        elif fault == "row":
            src[1] = ROWS
        elif fault == "page":
            table[src[2]][0] = PAGES
        elif fault == "order":
            keep[4][1] = keep[4][0]
        *self.want, bad = fork_reference(src, dst, n, table, pool, start, zero, PS)
        w_lens, w_table, w_shares, w_copies, w_counts = self.want
        self.want_caches = None
        if fault != "order":
            self.want_caches = [compact_reference(copy_reference(c, *w_copies), keep, list(map(len, keep)), [0] * ROWS, w_table)
                                for c in self.caches]
        ends = [r.randint(0, x) if x <= PS * WIDTH else 0 for x in w_lens]
        *self.want_free, bad_free = free_reference(w_lens, ends, w_table, pool, w_counts[0], w_shares, PS, PAGES)
        for t, x in ((self.src, src), (self.dst, dst), (self.lens, n), (self.table, table), (self.free, pool),
                     (self.start, [start]), (self.shares, zero), (self.ends, ends), (self.keep_lens, list(map(len, keep))),
                     (self.keep, [k + [0] * (8 - len(k)) for k in keep])):
            t.copy_(_i32(x))
        return not (bad or bad_free or fault == "order")

    def run(self):
        self.copies, self.counts = fa.paged_fork(self.src, self.dst, self.lens, self.table, self.free, self.shares, PS,
                                                 free_start=self.start)
        fa.paged_copy(self.copies[0], self.copies[1], *self.caches, rows=self.copies[2])
        fa.paged_compact(self.keep, self.keep_lens, self.base, self.table, *self.caches)
        self.freed = fa.paged_free(self.lens, self.ends, self.table, self.free, self.counts[:1], PS, PAGES,
                                   shares=self.shares)

    def compare(self):
        w_lens, w_table, w_shares, w_copies, w_counts = self.want
        w_free, w_shares, w_freed = self.want_free
        assert self.lens.tolist() == w_lens and self.table.tolist() == w_table
        assert self.copies.tolist() == w_copies and self.counts.tolist() == w_counts
        assert self.free.tolist() == w_free and self.shares.tolist() == w_shares and self.freed.tolist() == w_freed
        for c, w in zip(self.caches, self.want_caches or ()):
            assert torch.equal(bits(c), bits(w))


# a list with room for all, one without, and one that runs out of pages
STARTS = [36, 4, 40]
FAULTS = [None, None, "length", None, "row", "page", None, "order", None]


def test_status_of_replayed_steps(cuda_lib):
    s = Step(1)
    s.fill(36)
    s.run()
    _status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    seen = set()
    for start in STARTS:
        for fault in FAULTS:
            sound = s.fill(start, fault)
            seen.add((sound, fault))
            graph.replay()
            assert _status() == (_lib.FA_OK if sound else _lib.FA_ERR_INVALID_ARG), (start, fault)
            s.compare()
    assert (True, None) in seen and (False, None) in seen


def test_status_of_steps_on_two_streams(cuda_lib):
    """Both streams' calls set the one status of the device."""
    steps, streams = [Step(2), Step(3)], [torch.cuda.Stream() for _ in range(2)]
    seen = set()
    for start in STARTS:
        for fault in FAULTS:
            sound = [s.fill(start, f) for s, f in zip(steps, (fault, None))]
            seen.add(all(sound))
            torch.cuda.synchronize()
            for s, st in zip(steps, streams):
                with torch.cuda.stream(st):
                    s.run()
            assert _status() == (_lib.FA_OK if all(sound) else _lib.FA_ERR_INVALID_ARG), (start, fault, sound)
            for s in steps:
                s.compare()
    assert seen == {True, False}


@pytest.mark.parametrize("new", [[5, 2], [60, 2]])
def test_widest_window_is_sound(cuda_lib, new):
    r = random.Random(2)
    p = TreeProblem([random_tree(r, n, "any") for n in new], [n + 90 for n in new], 2, 1, 64, 16, BF)
    o, lse = fa.attention_fwd_paged_tree(p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), p.table.cuda(), _i32(p.lens),
                                         p.cu.cuda(), p.parents.cuda(), p.max_new, scale=p.scale, window=0x7FFFFFFF)
    assert _status() == _lib.FA_OK
    check(o, lse, p.reference(), p.rows)
