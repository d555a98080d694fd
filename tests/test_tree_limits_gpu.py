"""Trees of drafted tokens at the ends of their sizes, and the operators of
branching requests on several streams at once."""
import random

import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import check, pages_of
from _pages import free_reference
from _tree import TreeProblem, random_tree

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _tree(p, **kw):
    return fa.attention_fwd_paged_tree(p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), p.table.cuda(), _i32(p.lens),
                                       p.cu.cuda(), p.parents.cuda(), p.max_new, scale=p.scale, window=p.window or None,
                                       **kw)


@pytest.mark.parametrize("ctx,new,Hq,Hkv,d,ps,window", [
    ([3 + (7 * i) % 90 for i in range(700)], [1 + i % 4 for i in range(700)], 4, 2, 64, 16, 0),
    # more requests than have their tile counts kept in shared memory
    ([20 + (11 * i) % 150 for i in range(300)], [3 + (5 * i) % 17 for i in range(300)], 8, 1, 64, 16, 0),
    ([20 + (11 * i) % 150 for i in range(300)], [3 + (5 * i) % 17 for i in range(300)], 8, 1, 128, 32, 6),
    # few rows of most, and both kernels
    ([30 + (13 * i) % 400 for i in range(400)] + [300], [1 + (3 * i) % 4 for i in range(400)] + [200], 4, 1, 64, 16, 0),
    # blocks of up to 128 rows by turns with more: ranges cut amid a tile's units
    ([100, 130, 300, 1000, 513], [7, 20, 5, 30, 40], 4, 1, 128, 64, 0),
    ([1500, 900, 260, 1400], [9, 100, 60, 33], 8, 2, 128, 128, 0),
    ([2000, 100], [33, 70], 20, 4, 64, 16, 0),
    ([900, 80], [300, 20], 3, 3, 64, 32, 0),
    # a token's heads fill a tile, do not divide one, are more than a block
    ([300, 5], [2, 3], 128, 1, 64, 64, 0),
    ([300, 5], [3, 4], 200, 1, 64, 64, 2),
    ([200], [5], 300, 1, 128, 32, 0),
])
@pytest.mark.parametrize("cols", [1, 70])
def test_many_requests_and_wide_groups(cuda_lib, ctx, new, Hq, Hkv, d, ps, window, cols):
    r = random.Random(len(ctx))
    p = TreeProblem([random_tree(r, n, "any") for n in new], [c + n for c, n in zip(ctx, new)], Hq, Hkv, d, ps, BF, window,
                    extra_cols=cols)
    o, lse = _tree(p)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    check(o, lse, p.reference(), p.rows)


def test_a_quarter_billion_keys(cuda_lib):
    """100 drafted tokens that all follow a context of 230 million keys, for
    152 heads.  The table names 8 pages again and again, K is 0 and V is 1, so
    O is 1 (as for the causal rows: off by less than half a step of bf16) and
    every LSE the log of context + 1."""
    rows, heads, d, ps, keys = 100, 152, 64, 256, 230_000_000
    kc = torch.zeros(8, heads, ps, d, dtype=BF, device="cuda")
    vc = torch.ones_like(kc)
    table = (torch.arange(pages_of(keys, ps), dtype=torch.int32, device="cuda") % 8)[None].contiguous()
    q = torch.randn(rows, heads, d, device="cuda").to(BF)
    o, lse = fa.attention_fwd_paged_tree(q, kc, vc, table, _i32([keys]), _i32([0, rows]), _i32([-1] * rows), rows)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    want = torch.log(torch.tensor(keys - rows + 1.0, dtype=torch.float64, device="cuda"))
    assert (lse.double() - want).abs().max() <= 2.0 ** -22 * (1 + want) + 2.0 ** -23
    assert (o == 1).all()


@pytest.mark.parametrize("new", [[1024], [1000, 3]])
@pytest.mark.parametrize("window", [0, 700])
def test_longest_chain(cuda_lib, new, window):
    """The most rows of a request, each one's path all before it."""
    p = TreeProblem([random_tree(None, n, "chain") for n in new], [n + 40 for n in new], 1, 1, 64, 16, HF, window)
    o, lse = _tree(p)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    check(o, lse, p.reference(), p.rows)


def test_window_of_two_billion(cuda_lib):
    for new in ([5, 2], [60, 2]):
        r = random.Random(2)
        p = TreeProblem([random_tree(r, n, "any") for n in new], [n + 90 for n in new], 2, 1, 64, 16, BF)
        want = p.reference()
        p.window = 0x7FFFFFFF
        check(*_tree(p), want, p.rows)


def test_free_of_a_cluster_captured_and_on_two_streams(cuda_lib):
    """Calls large enough for sixteen CTAs, each of a pool of its own, at once."""
    r = random.Random(9)
    calls = []
    for seed in range(2):
        B, top = 1200, 16 * 60
        old = [r.randint(0, top) for _ in range(B)]
        new = [r.choice([0, r.randint(0, n)]) for n in old]
        ids = list(range(sum(pages_of(n, 16) for n in old)))
        num = len(ids)
        r.shuffle(ids)
        table = [[ids.pop() if c < pages_of(n, 16) else -1 for c in range(60)] for n in old]
        shares = [0] * num
        for b in range(1, B, 2):
            for c in range(min(pages_of(old[b], 16), pages_of(old[b - 1], 16)) // 2):
                table[b][c] = table[b - 1][c]
                shares[table[b][c]] = 1
        want = free_reference(old, new, table, [-1] * num, num, shares, 16, num)
        assert not want[3]
        calls.append((want, _i32(shares), _i32(old), _i32(new), torch.tensor(table, dtype=torch.int32, device="cuda"),
                      _i32([-1] * num), _i32([num]), num, torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for want, shares0, old, new, table, free, start, num, st in calls:
        shares = shares0.clone()
        with torch.cuda.stream(st):
            st.wait_stream(torch.cuda.default_stream())
            fa.paged_free(old, new, table, free, start, 16, num, shares=shares)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            shares.copy_(shares0)
            counts = fa.paged_free(old, new, table, free, start, 16, num, shares=shares)
        graphs.append((g, st, free, shares, counts, want))
    for turn in range(3):
        for g, st, free, shares, counts, want in graphs:
            free.fill_(-1)
        torch.cuda.synchronize()
        for g, st, *_ in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert _lib.fa_get_device_status() == _lib.FA_OK
        for g, st, free, shares, counts, want in graphs:
            assert free.tolist() == want[0] and shares.tolist() == want[1] and counts.tolist() == want[2]


def test_operators_overlap_on_streams(cuda_lib):
    """The four operators behind one another on two streams, pools apart."""
    from _pages import bits, compact_reference, copy_reference, fork_reference
    r = random.Random(4)
    jobs = []
    for seed in range(2):
        g = torch.Generator("cuda").manual_seed(seed)
        caches = [torch.randint(-32768, 32768, (300, 2, 32, 128), generator=g, device="cuda", dtype=torch.int16).view(BF)
                  for _ in range(2)]
        ids = r.sample(range(300), 300)
        table = [[ids.pop() for _ in range(8)] for _ in range(12)] + [[-1] * 8 for _ in range(12)]
        lens = [r.randint(1, 250) for _ in range(12)] + [0] * 12
        src, dst = [r.randrange(6) for _ in range(12)], list(range(12, 24))
        free, start, shares = ids[:100], 20, [0] * 300
        w_lens, w_table, w_shares, w_copies, w_counts, bad = fork_reference(src, dst, lens, table, free, start, shares, 32)
        keep = [sorted(r.sample(range(n), n // 2)) if 6 <= b < 12 else [] for b, n in enumerate(w_lens)]
        w_caches = [compact_reference(copy_reference(c, *w_copies), keep, list(map(len, keep)), [0] * 24, w_table)
                    for c in caches]
        ends = [0 if b % 3 == 0 else n // 2 for b, n in enumerate(w_lens)]
        w_free, w_shares, w_freed, _ = free_reference(w_lens, ends, w_table, free, w_counts[0], w_shares, 32, 300)
        most = max(1, max(map(len, keep)))
        jobs.append(dict(st=torch.cuda.Stream(), caches=caches, lens=_i32(lens), free=_i32(free), shares=_i32(shares),
                         table=torch.tensor(table, dtype=torch.int32, device="cuda"), src=_i32(src), dst=_i32(dst),
                         start=_i32([start]), ends=_i32(ends), keep_lens=_i32(map(len, keep)), base=_i32([0] * 24),
                         keep=torch.tensor([k + [0] * (most - len(k)) for k in keep], dtype=torch.int32, device="cuda"),
                         want=(w_lens, w_table, w_shares, w_copies, w_counts, w_free, w_freed, w_caches)))
    torch.cuda.synchronize()
    for j in jobs:
        with torch.cuda.stream(j["st"]):
            j["copies"], j["counts"] = fa.paged_fork(j["src"], j["dst"], j["lens"], j["table"], j["free"], j["shares"], 32,
                                                     free_start=j["start"])
            fa.paged_copy(j["copies"][0], j["copies"][1], *j["caches"], rows=j["copies"][2])
            fa.paged_compact(j["keep"], j["keep_lens"], j["base"], j["table"], *j["caches"])
            j["freed"] = fa.paged_free(j["lens"], j["ends"], j["table"], j["free"], j["counts"][:1], 32, 300,
                                       shares=j["shares"])
    torch.cuda.synchronize()
    _lib.fa_get_device_status()  # a list without room for all is reported
    for j in jobs:
        w_lens, w_table, w_shares, w_copies, w_counts, w_free, w_freed, w_caches = j["want"]
        assert j["lens"].tolist() == w_lens and j["table"].tolist() == w_table and j["shares"].tolist() == w_shares
        assert j["copies"].tolist() == w_copies and j["counts"].tolist() == w_counts
        assert j["free"].tolist() == w_free and j["freed"].tolist() == w_freed
        for c, w in zip(j["caches"], w_caches):
            assert torch.equal(bits(c), bits(w))
