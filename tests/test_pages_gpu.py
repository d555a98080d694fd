"""Forking, copying, compacting and freeing pages of a cache, against
references that go request by request (_pages): every output is a whole number
or a moved value, so all of them have to be equal."""
import random

import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import pages_of
from _pages import bits, compact_reference, copy_reference, fork_reference, free_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _status():
    torch.cuda.synchronize()
    return _lib.fa_get_device_status()


def _table(r, lens, ps, width, extra=0):
    """Distinct pages for every request's tokens, numbers outside the pool
    behind them; (table, pool size, pages left over)."""
    num = sum(pages_of(n, ps) for n in lens) + extra
    ids = list(range(num))
    r.shuffle(ids)
    return [[ids.pop() if c < pages_of(n, ps) else num + 5 for c in range(width)] for n in lens], num, ids


# -------------------------------------------------------------------- fork


def _fork(src, dst, lens, table, free, start, shares, ps, unsound=False):
    want = fork_reference(src, dst, lens, table, free, start, shares, ps)
    g_lens, g_table, g_shares = _i32(lens), _i32(table), _i32(shares)
    copies, counts = fa.paged_fork(_i32(src), _i32(dst), g_lens, g_table, _i32(free), g_shares, ps,
                                   free_start=_i32([start]))
    assert _status() == (_lib.FA_ERR_INVALID_ARG if want[5] else _lib.FA_OK)
    assert want[5] == unsound
    got = (g_lens.tolist(), g_table.tolist(), g_shares.tolist(), copies.tolist(), counts.tolist())
    for a, b, what in zip(got, want, ("lens", "table", "shares", "copies", "counts")):
        assert a == b, what


@pytest.mark.parametrize("lens,forks,ps,width,spare", [
    ([1], 1, 16, 1, 1),
    ([0], 3, 16, 4, 2),                     # a row without tokens
    ([16], 2, 16, 1, 0),                    # full pages only: nothing to take
    ([17, 32, 15], 7, 16, 3, 9),
    ([2000], 8, 64, 40, 8),
    ([300, 5, 0, 64, 65], 23, 32, 10, 30),
    ([5000, 4097, 4096, 1], 9, 16, 333, 12),  # several units of cells a row
    ([90] * 40, 400, 16, 6, 400),
    ([77] * 3, 50, 16, 5, 20),              # a pool that runs out on the way
    ([40, 48, 33], 30, 16, 3, 0),           # and one that is empty
    ([700], 2500, 16, 50, 2500),            # more forks of a row than a block has threads
])
def test_fork(cuda_lib, lens, forks, ps, width, spare):
    r = random.Random(len(lens) + forks)
    table, num, free = _table(r, lens, ps, width, spare + 3)
    table += [[num + 9] * width for _ in range(forks + 2)]
    rows = list(range(len(table)))
    r.shuffle(rows)
    shuffled = [None] * len(rows)
    all_lens = [0] * len(rows)
    for i, at in enumerate(rows):
        shuffled[at] = table[i]
        all_lens[at] = lens[i] if i < len(lens) else 7 * i % 11
    src = [rows[r.randrange(len(lens))] for _ in range(forks)]
    dst = rows[len(lens):len(lens) + forks]
    free = free[:spare + 3]
    _fork(src, dst, all_lens, shuffled, free, min(3, len(free)), [i % 3 for i in range(num)], ps)


def test_fork_of_shared_pages(cuda_lib):
    """Two rows that name the same pages branch in one call."""
    table = [[4, 1, 0], [4, 1, 2], [9, 9, 9], [9, 9, 9], [9, 9, 9]]
    _fork([0, 1, 0], [2, 3, 4], [40, 48, 0, 0, 0], table, [3, 5], 0, [0, 1, 0, 0, 1, 0], 16)


def test_fork_reports_unsound(cuda_lib):
    table = [[0, 1], [2, 99], [9, 9], [9, 9], [9, 9], [-4, 3], [9, 9]]
    lens = [20, 32, 5, 6, 7, 20, 8]
    free = [10, 11, 77, 12]
    # rows outside the table, a row onto itself, a length beyond the row; sound ones beside them
    _fork([0, -1, 0, 2, 0], [2, 3, 7, 2, 4], lens, table, free, 0, [0] * 16, 16, True)
    _fork([0, 0], [2, 3], [33, 0, 0, 0, 0, 0, 0], table, free, 0, [0] * 16, 16, True)
    _fork([0, 0], [2, 3], [-1, 0, 0, 0, 0, 0, 0], table, free, 0, [0] * 16, 16, True)
    # pages outside the pool: in a shared cell, in a copied one, in the free list
    _fork([1, 5, 0, 0], [2, 3, 4, 6], lens[:1] + [32] + lens[2:], table, free, 0, [0] * 16, 16, True)


def test_fork_start_outside_the_list(cuda_lib):
    lens, table, shares = _i32([20, 0]), _i32([[0, 1], [5, 5]]), _i32([0] * 4)
    copies, counts = fa.paged_fork(_i32([0]), _i32([1]), lens, table, _i32([2]), shares, 16, free_start=_i32([3]))
    assert _status() == _lib.FA_ERR_INVALID_ARG
    assert lens.tolist() == [20, 0] and table.tolist() == [[0, 1], [5, 5]] and copies.flatten().tolist() == [-1, -1, 0]


def test_fork_most(cuda_lib):
    n, ps = 8192, 16
    r = random.Random(3)
    table, num, free = _table(r, [40] * 8, ps, 3, n)
    table += [[num] * 3 for _ in range(n)]
    _fork([r.randrange(8) for _ in range(n)], list(range(8, 8 + n)), [40] * 8 + [0] * n, table, free, 0, [0] * num, ps)
    with pytest.raises(_lib.FAError) as e:
        big = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        fa.paged_fork(big, big.clone(), torch.zeros(n + 9, dtype=torch.int32, device="cuda"),
                      torch.zeros(n + 9, 3, dtype=torch.int32, device="cuda"), big.clone(), big.clone(), ps)
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED


# -------------------------------------------------------------------- copy


def _caches(pages, Hkv, ps, d, dtype, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    # any 16 bits: NaN and infinities are moved like the rest
    return [torch.randint(-32768, 32768, (pages, Hkv, ps, d), generator=g, device="cuda", dtype=torch.int16).view(dtype)
            for _ in range(2)]


@pytest.mark.parametrize("Hkv,ps,d,dtype", [(1, 16, 64, BF), (2, 16, 128, HF), (8, 64, 128, BF), (3, 256, 64, HF),
                                            (5, 256, 128, BF), (7, 32, 64, HF), (1, 128, 128, BF)])
@pytest.mark.parametrize("n", [1, 2, 37])
def test_copy(cuda_lib, Hkv, ps, d, dtype, n):
    r = random.Random(n * Hkv + ps)
    caches = _caches(2 * n + 3, Hkv, ps, d, dtype)
    ids = list(range(2 * n + 3))
    r.shuffle(ids)
    src, dst = [ids[i // 2 * 2] for i in range(n)], ids[n + 1:2 * n + 1]  # a source may occur twice
    dst = [p if p not in src else -1 for p in dst]
    if n > 5:
        src[3], dst[5] = -1, -7
    for rows in (None, [r.choice([0, 1, ps - 1, ps, r.randint(0, ps)]) for _ in range(n)]):
        want = [copy_reference(c, src, dst, rows or [ps] * n) for c in caches]
        fa.paged_copy(_i32(src), _i32(dst), *caches, rows=None if rows is None else _i32(rows))
        assert _status() == _lib.FA_OK
        for c, w in zip(caches, want):
            assert torch.equal(bits(c), bits(w))


def test_copy_reports_unsound(cuda_lib):
    caches = _caches(6, 2, 16, 64, BF)
    src, dst, rows = [0, 6, 1, 2, 3], [4, 5, 1 << 30, 5, 2], [16, 16, 16, 17, -1]
    want = [copy_reference(c, [0], [4], [16]) for c in caches]
    fa.paged_copy(_i32(src), _i32(dst), *caches, rows=_i32(rows))
    assert _status() == _lib.FA_ERR_INVALID_ARG
    for c, w in zip(caches, want):
        assert torch.equal(bits(c), bits(w))


# ----------------------------------------------------------------- compact


def _compact(lens, base, keep, Hkv, ps, d, dtype, max_keep=None, seed=0):
    r = random.Random(seed)
    width = max(1, max(pages_of(n, ps) for n in lens))
    table, num, _ = _table(r, lens, ps, width, 2)
    caches = _caches(num, Hkv, ps, d, dtype, seed)
    want = [compact_reference(c, keep, [len(k) for k in keep], base, table) for c in caches]
    most = max(1, max(len(k) for k in keep)) if max_keep is None else max_keep
    # entries behind a request's are not read
    g_keep = _i32([k + [-9] * (most - len(k)) for k in keep])
    fa.paged_compact(g_keep, _i32([len(k) for k in keep]), _i32(base), _i32(table), *caches)
    assert _status() == _lib.FA_OK
    for c, w in zip(caches, want):
        assert torch.equal(bits(c), bits(w))


@pytest.mark.parametrize("Hkv,ps,d,dtype", [(1, 16, 64, BF), (2, 16, 128, HF), (8, 64, 128, BF), (3, 256, 64, HF)])
def test_compact_small(cuda_lib, Hkv, ps, d, dtype):
    # nothing, all, the first, the last, places that are both read and written, pages' borders
    _compact([1, 30, 5, 64, 40, 33, 17], [0, 10, 5, 0, 7, 15, 16],
             [[0], [0, 3, 4, 9, 19], [], list(range(64)), list(range(1, 33)), [17], [0]], Hkv, ps, d, dtype)


@pytest.mark.parametrize("seed", range(16))
def test_compact_random(cuda_lib, seed):
    r = random.Random(seed)
    ps, d, Hkv = r.choice([16, 32, 64, 128, 256]), r.choice([64, 128]), r.choice([1, 2, 3, 4, 8])
    B = r.choice([1, 2, 9, 40])
    lens = [r.choice([r.randint(1, 20), r.randint(1, 3000 if B < 9 else 400)]) for _ in range(B)]
    base = [r.choice([0, r.randint(0, n)]) for n in lens]
    keep = []
    for n, b in zip(lens, base):
        m = r.choice([0, n - b, r.randint(0, n - b), min(5, n - b)])
        keep.append(sorted(r.sample(range(n - b), m)))
    _compact(lens, base, keep, Hkv, ps, d, r.choice([BF, HF]), seed=seed)


@pytest.mark.parametrize("Hkv,d,B", [(1, 64, 1), (1, 128, 1), (2, 128, 3), (4, 64, 30), (8, 128, 20)])
def test_compact_long_shifts_by_one(cuda_lib, Hkv, d, B):
    """Every place is read and written: with 1, 2, 4 and 8 blocks a row."""
    n = 4100
    _compact([n] * B, [0] * B, [list(range(1, n)) for _ in range(B)], Hkv, 64, d, BF, max_keep=n + 3)


def test_compact_reports_unsound(cuda_lib):
    table = [[0, 1], [2, 3], [4, 5], [6, 99], [7, -1], [8, 9], [10, 11], [12, 13]]
    caches = _caches(16, 2, 16, 64, BF)
    keep = [[1, 3], [1, 1], [-1, 4], [0, 20], [17, 18], [2, 40], [3, 4], [5, 9]]
    keep_lens, base = [2, 2, 2, 2, 2, 2, 3, 2], [0, 0, 0, 0, 0, 0, 0, 33]
    want = [compact_reference(c, [[1, 3], [1], [0, 4], [0], [], [2]], [2, 1, 2, 1, 0, 1], [0] * 6, table)
            for c in caches]
    fa.paged_compact(_i32(keep), _i32(keep_lens), _i32(base), _i32(table), *caches)
    assert _status() == _lib.FA_ERR_INVALID_ARG
    for c, w in zip(caches, want):
        assert torch.equal(bits(c), bits(w))


# -------------------------------------------------------------------- free


def _free(old, new, table, free, start, shares, ps, num_pages, unsound=False):
    want = free_reference(old, new, table, free, start, shares, ps, num_pages)
    g_free, g_shares = _i32(free), None if shares is None else _i32(shares)
    counts = fa.paged_free(_i32(old), _i32(new), _i32(table), g_free, _i32([start]), ps, num_pages, shares=g_shares)
    assert _status() == (_lib.FA_ERR_INVALID_ARG if want[3] else _lib.FA_OK)
    assert want[3] == unsound
    assert counts.tolist() == want[2]
    assert g_free.tolist() == want[0]
    if shares is not None:
        assert g_shares.tolist() == want[1]


@pytest.mark.parametrize("seed", range(20))
def test_free_random(cuda_lib, seed):
    r = random.Random(seed)
    ps = r.choice([16, 32, 64, 128, 256])
    B = r.choice([1, 2, 7, 33, 300])
    top = r.choice([1, ps, 3 * ps, 3000])
    old = [r.choice([0, r.randint(0, top), top]) for _ in range(B)]
    new = [r.choice([0, n, r.randint(0, n), max(0, n - 1)]) for n in old]
    table, num, spare = _table(r, old, ps, pages_of(top, ps) + r.choice([0, 1, 50]), 9)
    start = num - len(spare)
    _free(old, new, table, [-1] * start + spare, start, None, ps, num)
    # pages of several requests: rows that begin like another one
    shares = [0] * num
    for b in range(1, B):
        o = r.randrange(b)
        for c in range(r.randint(0, min(pages_of(old[o], ps), pages_of(old[b], ps)))):
            if shares[table[b][c]] == 0 and table[b][c] != table[o][c]:
                table[b][c] = table[o][c]
                shares[table[o][c]] += 1
    _free(old, new, table, [-1] * start + spare, start, shares, ps, num)


@pytest.mark.parametrize("B,tokens", [(1, 16 * 9000), (500, 16 * 100), (16384, 40), (3000, 16 * 120)])
def test_free_many(cuda_lib, B, tokens):
    r = random.Random(B)
    old = [tokens] * B
    table, num, spare = _table(r, old, 16, pages_of(tokens, 16), 2)
    start = num - 2
    _free(old, [0] * B, table, [-3] * start + spare, start, None, 16, num)
    # all pages of the odd rows are those of the even ones; every third row stays
    for b in range(1, B, 2):
        table[b] = table[b - 1]
    shares = [0] * num
    for b in range(0, B - 1, 2):
        for p in table[b]:
            shares[p] = 1
    _free(old, [tokens - 20 if b % 3 == 0 else 0 for b in range(B)], table, [-3] * start + spare, start, shares, 16, num)


def test_free_page_given_up_more_often_than_held(cuda_lib):
    _free([48, 48], [0, 0], [[3, 3, 1], [1, 2, 3]], [7] * 9, 6, [0] * 5, 16, 5)


def test_free_without_room(cuda_lib):
    _free([64, 40], [16, 0], [[3, 4, 5, 6], [0, 1, 2, 9]], [7] * 6, 4, [0] * 8, 16, 8, True)
    _free([64, 40], [16, 0], [[3, 4, 5, 6], [0, 1, 2, 9]], [7] * 6, 0, None, 16, 8, True)
    # nothing is freed: an empty list is as good
    _free([64, 40], [60, 33], [[3, 4, 5, 6], [0, 1, 2, 9]], [], 0, None, 16, 8)


def test_free_reports_unsound(cuda_lib):
    table = [[3, 4], [5, 99], [0, 1], [2, 6], [7, -1], [8, 9]]
    for shares in (None, [0, 0, 1, 0, 0, 0, 0, 0, 0, 0]):
        _free([32, 32, 33, 32, 20, 16], [0, 0, 0, -1, 3, 17], table, [7] * 9, 8, shares, 16, 10, True)


def test_free_start_outside_the_list(cuda_lib):
    for start in (-1, 4):
        free = _i32([5, 6, 7])
        counts = fa.paged_free(_i32([16]), _i32([0]), _i32([[1]]), free, _i32([start]), 16, 8)
        assert _status() == _lib.FA_ERR_INVALID_ARG
        assert free.tolist() == [5, 6, 7] and counts.tolist() == [0, 1]


# ------------------------------------------------------- together, captured


def test_pool_through_a_life(cuda_lib):
    """Prompts, samples of them, drafted tokens of which some stay, ends: the
    pool's pages are all there in the end, each once, and the caches hold what
    lists of tokens say."""
    ps, Hkv, d, B, num = 16, 2, 64, 12, 120
    r = random.Random(5)
    k_cache, v_cache = (torch.zeros(num, Hkv, ps, d, dtype=BF, device="cuda") for _ in range(2))
    free = _i32(r.sample(range(num), num))
    start, shares = _i32([0]), _i32([0] * num)
    table, lens = _i32([[-1] * 16 for _ in range(B)]), _i32([0] * B)
    truth, count = [[] for _ in range(B)], 0

    def append(new):
        nonlocal lens, start, count
        total = max(1, sum(new))
        after, cu, slots, counts = fa.paged_tables(lens, _i32(new), table, free, ps, num, total, free_start=start)
        rows = []
        for b, n in enumerate(new):
            mine = list(range(count, count + n))
            count += n
            truth[b] += mine
            rows += mine
        x = torch.tensor(rows or [0], device="cuda")[:, None, None].expand(total, Hkv, d)
        fa.paged_append((x % 128).to(BF).contiguous(), (x // 128).to(BF).contiguous(), slots, k_cache, v_cache)
        lens, start = after, counts[:1].clone()

    append([37, 64] + [0] * (B - 2))
    src, dst = _i32([0, 1, 0, 1, 0]), _i32([2, 3, 4, 5, 6])
    copies, counts = fa.paged_fork(src, dst, lens, table, free, shares, ps, free_start=start)
    fa.paged_copy(copies[0], copies[1], k_cache, v_cache, rows=copies[2])
    start = counts[:1].clone()
    for s, t in zip(src.tolist(), dst.tolist()):
        truth[t] = list(truth[s])
    for step in range(6):
        before = lens.tolist()
        new = [r.randint(0, 20) if b < 7 else 0 for b in range(B)]
        append(new)
        keep = [sorted(r.sample(range(n), r.randint(0, n))) for n in new]
        fa.paged_compact(_i32([k + [0] * (20 - len(k)) for k in keep]), _i32([len(k) for k in keep]), _i32(before), table,
                         k_cache, v_cache)
        for b, k in enumerate(keep):
            truth[b] = truth[b][:before[b]] + [truth[b][before[b] + i] for i in k]
        after = [n + len(k) for n, k in zip(before, keep)]
        if step == 3:  # a prompt's own row ends before its samples
            after[0], truth[0] = 0, []
        counts = fa.paged_free(lens, _i32(after), table, free, start, ps, num, shares=shares)
        lens, start = _i32(after), counts[:1].clone()
        assert _status() == _lib.FA_OK
        for b, tokens in enumerate(truth):
            got = [int(k_cache[table[b, t // ps], 1, t % ps, 3]) + 128 * int(v_cache[table[b, t // ps], 0, t % ps, 60])
                   for t in range(len(tokens))]
            assert got == tokens, (step, b)
    counts = fa.paged_free(lens, _i32([0] * B), table, free, start, ps, num, shares=shares)
    assert _status() == _lib.FA_OK
    assert counts.tolist() == [0, 0] and sorted(free.tolist()) == list(range(num)) and not any(shares.tolist())


def test_captured_and_replayed(cuda_lib):
    """Fork, copy, compact and free in one graph, replayed as its inputs change in place."""
    ps, num, width = 16, 40, 6
    r = random.Random(1)
    caches = _caches(num, 2, ps, 128, HF)
    src, dst = _i32([0, 0]), _i32([2, 3])
    lens, table = _i32([0] * 4), _i32([[0] * width for _ in range(4)])
    free, start, shares = _i32([0] * 20), _i32([0]), _i32([0] * num)
    keep, keep_lens, base, new = _i32([[0] * 8 for _ in range(4)]), _i32([0] * 4), _i32([0] * 4), _i32([0] * 4)
    out = {}

    def step():
        out["copies"], out["counts"] = fa.paged_fork(src, dst, lens, table, free, shares, ps, free_start=start)
        fa.paged_copy(out["copies"][0], out["copies"][1], *caches, rows=out["copies"][2])
        fa.paged_compact(keep, keep_lens, base, table, *caches)
        out["freed"] = fa.paged_free(lens, new, table, free, out["counts"][:1], ps, num, shares=shares)

    step()
    assert _status() == _lib.FA_OK
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        n = [r.randint(1, 80), r.randint(1, 80), 0, 0]
        pages = r.sample(range(num), num)
        rows = [[pages.pop() for _ in range(width)] for _ in range(2)] + [[-1] * width] * 2
        pool = (pages + [0] * 20)[:20]
        s, zero = [r.randrange(2), r.randrange(2)], [0] * num
        w_lens, w_table, w_shares, w_copies, w_counts, bad = fork_reference(s, [2, 3], n, rows, pool, 4, zero, ps)
        assert not bad
        own = [b for b in range(2) if b not in s]  # a row whose pages are its own moves tokens
        k = [sorted(r.sample(range(n[b]), min(8, n[b] // 2))) if b in own else [] for b in range(4)]
        w_caches = [copy_reference(c, *w_copies) for c in caches]
        w_caches = [compact_reference(c, k, [len(x) for x in k], [0] * 4, w_table) for c in w_caches]
        ends = [r.randint(0, x) for x in w_lens]
        w_free, w_shares, w_freed, bad = free_reference(w_lens, ends, w_table, pool, w_counts[0], w_shares, ps, num)
        assert not bad or w_freed[1]
        for t, x in ((src, s), (lens, n), (table, rows), (free, pool), (start, [4]), (shares, zero), (new, ends),
                     (keep, [x + [0] * (8 - len(x)) for x in k]), (keep_lens, [len(x) for x in k])):
            t.copy_(_i32(x))
        graph.replay()
        _status()
        assert lens.tolist() == w_lens and table.tolist() == w_table and out["copies"].tolist() == w_copies
        assert out["counts"].tolist() == w_counts and out["freed"].tolist() == w_freed
        assert free.tolist() == w_free and shares.tolist() == w_shares
        for c, w in zip(caches, w_caches):
            assert torch.equal(bits(c), bits(w))


def test_on_a_named_stream(cuda_lib):
    st = torch.cuda.Stream()
    caches = _caches(8, 1, 16, 64, BF)
    want = [copy_reference(c, [1], [6], [5]) for c in caches]
    lens, table, shares = _i32([21, 0]), _i32([[0, 1], [0, 0]]), _i32([0] * 8)
    args = _i32([0]), _i32([1]), lens, table, _i32([6]), shares, 16
    st.wait_stream(torch.cuda.current_stream())
    copies, counts = fa.paged_fork(*args, stream=st)
    fa.paged_copy(copies[0], copies[1], *caches, rows=copies[2], stream=st)
    freed = fa.paged_free(lens, torch.zeros_like(lens), table, _i32([0] * 3), _i32([3]), 16, 8, shares=shares,
                          stream=st.cuda_stream)
    st.synchronize()
    assert copies.flatten().tolist() == [1, 6, 5] and counts.tolist() == [1, 0] and freed.tolist() == [0, 0]
    for c, w in zip(caches, want):
        assert torch.equal(bits(c), bits(w))


def test_offsets_past_32_bits(cuda_lib):
    """Caches of more than 2^32 values: their last pages."""
    Hkv, ps, d = 8, 256, 128
    num = (1 << 32) // (Hkv * ps * d) + 40
    k_cache, v_cache = (torch.zeros(num, Hkv, ps, d, dtype=BF, device="cuda") for _ in range(2))
    rows = torch.randn(2, Hkv, ps, d, device="cuda").to(BF)
    k_cache[num - 3], v_cache[num - 3] = rows[0], rows[1]
    fa.paged_copy(_i32([num - 3]), _i32([num - 1]), k_cache, v_cache)
    fa.paged_compact(_i32([[5, 9, 200]]), _i32([3]), _i32([3]), _i32([[num - 1]]), k_cache, v_cache)
    assert _status() == _lib.FA_OK
    at = torch.arange(ps)
    at[3:6] = torch.tensor([8, 12, 203])
    for c, x in ((k_cache, rows[0]), (v_cache, rows[1])):
        assert torch.equal(c[num - 1], x[:, at]) and torch.equal(c[num - 3], x)
        assert not c[num - 2].any() and not c[0].any()


def test_python_refusals(cuda_lib):
    i = _i32([0])
    caches = _caches(4, 1, 16, 64, BF)
    table = _i32([[0, 1]])
    for bad in (i.long(), i.cpu(), _i32([[0, 1], [2, 3]])[:, 0]):
        with pytest.raises((TypeError, ValueError)):
            fa.paged_copy(bad, i, *caches)
        with pytest.raises((TypeError, ValueError)):
            fa.paged_free(bad, i, table, i.clone(), _i32([1]), 16, 4)
        with pytest.raises((TypeError, ValueError)):
            fa.paged_fork(bad, i, i.clone(), table, i.clone(), i.clone(), 16)
        with pytest.raises((TypeError, ValueError)):
            fa.paged_compact(_i32([[0]]), bad, i, table, *caches)
    with pytest.raises(ValueError):
        fa.paged_copy(i, i.clone(), caches[0], caches[1][:2])
    with pytest.raises(ValueError):
        fa.paged_copy(i, _i32([1, 2]), *caches)
    with pytest.raises((TypeError, ValueError)):
        fa.paged_copy(i, i.clone(), caches[0], caches[1].to(HF))
    with pytest.raises(TypeError):
        fa.paged_copy(i, i.clone(), *(c.view(torch.int16) for c in caches))
    with pytest.raises(ValueError):
        fa.paged_compact(_i32([0]), i, i, table, *caches)
    with pytest.raises(ValueError):
        fa.paged_free(i, i, table, i.clone(), _i32([1]), 16, 4, shares=_i32([0] * 5))
    with pytest.raises(ValueError):
        fa.paged_free(i, i, table, i.clone(), _i32([1]), 1 << 40, 4)
    assert _status() == _lib.FA_OK
