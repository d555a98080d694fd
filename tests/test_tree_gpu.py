"""Attention of trees of drafted tokens against a plain form in 64 bits."""
import random

import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import check
from _tree import TreeProblem, path_of, random_tree

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _args(p):
    return [p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), p.table.cuda(), _i32(p.lens), p.cu.cuda(), p.parents.cuda()]


def _run(p, **kw):
    kw = {"max_new": p.max_new, **kw}
    o, lse = fa.attention_fwd_paged_tree(*_args(p), scale=p.scale, window=p.window or None, **kw)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    return o, lse


# context, drafted tokens, kind of tree, Hq, Hkv, d, page_size, dtype, window
CASES = [
    # up to 16 rows a key/value head: lengths around tiles and pages
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 300], [1, 2, 3, 4, 5, 6, 7, 8, 16, 9, 12], "any", 2, 2, 128, 16, BF, 0),
    ([60, 62, 126, 127, 128, 1000], [8] * 6, "near", 4, 2, 64, 64, HF, 0),
    ([333], [8], "any", 16, 16, 128, 64, BF, 0),
    ([500, 3], [4, 4], "star", 8, 2, 128, 32, HF, 0),
    ([257, 90], [16, 16], "comb", 3, 3, 64, 256, BF, 0),
    ([7, 1200], [2, 5], "chain", 6, 2, 128, 128, BF, 0),
    # more
    ([0, 1, 100, 128, 1000], [17, 33, 64, 128, 129], "any", 4, 1, 128, 64, BF, 0),
    ([333, 64, 65], [256, 257, 63], "any", 2, 1, 64, 16, HF, 0),
    ([700, 20], [64, 60], "star", 8, 2, 128, 128, HF, 0),
    ([5, 250], [300, 20], "near", 3, 1, 128, 32, BF, 0),
    ([100, 1030], [40, 63], "comb", 5, 1, 64, 64, BF, 0),
    ([200], [1024], "any", 1, 1, 64, 16, BF, 0),
    ([77], [600], "chain", 2, 1, 128, 256, HF, 0),
    # few rows of most requests, many of some: both kernels
    ([400, 90, 1, 700, 64, 0, 129, 1500, 33], [200, 1, 1, 2, 4, 0, 3, 1, 4], "any", 8, 2, 128, 16, BF, 0),
    ([900, 10, 2000, 77, 65, 300, 8, 1], [260, 4, 1, 5, 1, 2, 8, 1], "near", 4, 2, 64, 64, HF, 0),
    # windows: within the path, at its end, in the context, wider than all
    ([500, 20, 129], [8, 8, 8], "near", 4, 2, 128, 16, BF, 3),
    ([500, 20, 129], [8, 5, 8], "any", 2, 2, 64, 64, HF, 1),
    ([500, 20, 129], [4, 2, 4], "chain", 4, 1, 128, 32, BF, 100),
    ([900, 300, 1], [100, 7, 40], "near", 4, 1, 128, 32, BF, 64),
    ([900, 300, 64], [150, 200, 33], "chain", 2, 1, 64, 16, HF, 20),
    ([900, 300, 64], [150, 200, 33], "any", 3, 1, 128, 64, BF, 2),
    ([600], [700], "near", 1, 1, 64, 128, HF, 300),
    ([100, 200], [50, 60], "any", 4, 2, 128, 16, BF, 5000),
    ([400, 90, 1, 700, 64, 0, 129, 1500, 33], [200, 1, 1, 2, 4, 0, 3, 1, 4], "near", 8, 2, 64, 16, HF, 40),
]


@pytest.mark.parametrize("ctx,new,kind,Hq,Hkv,d,ps,dtype,window", CASES)
@pytest.mark.parametrize("cols", [1, 80])  # a wide table may hold long sequences: their keys are split
def test_tree_matches_64_bits(cuda_lib, ctx, new, kind, Hq, Hkv, d, ps, dtype, window, cols):
    r = random.Random(len(ctx) + d)
    p = TreeProblem([random_tree(r, n, kind) for n in new], [c + n for c, n in zip(ctx, new)], Hq, Hkv, d, ps, dtype,
                    window, seed=d + ps, extra_cols=cols)
    check(*_run(p), p.reference(), p.rows)


@pytest.mark.parametrize("seed", range(30))
def test_tree_random(cuda_lib, seed):
    r = random.Random(seed)
    Hkv, group, d = r.choice([1, 2, 3, 4]), r.choice([1, 2, 3, 5, 7, 8, 16, 24]), r.choice([64, 128])
    B = r.choice([1, 2, 5, 9])
    most = r.choice([1, 4, 12, 40, 130])
    new = [r.randint(0, most) for _ in range(B)]
    new[r.randrange(B)] = most
    lens = [n + r.choice([0, r.randint(0, 60), r.randint(0, 700)]) for n in new]
    kind = r.choice(["chain", "star", "comb", "near", "any", "any"])
    p = TreeProblem([random_tree(r, n, kind) for n in new], lens, Hkv * group, Hkv, d, r.choice([16, 32, 64, 128, 256]),
                    r.choice([BF, HF]), r.choice([0, 0, r.randint(1, 8), r.randint(1, 300)]), seed=seed,
                    pad_rows=r.choice([0, 3]), sharp=r.choice([1.0, 4.0]), extra_cols=r.choice([1, 100]))
    o, lse = _run(p, max_new=p.max_new + r.choice([0, 0, 50]))
    check(o, lse, p.reference(), p.rows)


@pytest.mark.parametrize("lens,new,kind,window", [
    ([3, 0, 40], [5, 2, 1], "any", 0), ([2], [100], "near", 0), ([5, 60], [20, 70], "chain", 3), ([0], [1], "star", 0),
])
def test_tree_of_more_rows_than_keys(cuda_lib, lens, new, kind, window):
    """No context: the first drafted tokens have no keys."""
    r = random.Random(1)
    p = TreeProblem([random_tree(r, n, kind) for n in new], lens, 4, 2, 64, 16, HF, window)
    check(*_run(p), p.reference(), p.rows)


@pytest.mark.parametrize("new,Hq,Hkv,d,window", [([4, 1, 3], 8, 2, 128, 0), ([4, 1, 3], 4, 2, 64, 50),
                                                 ([300, 17], 2, 1, 128, 0), ([90, 100], 4, 1, 64, 200)])
def test_chain_is_the_causal_forward(cuda_lib, new, Hq, Hkv, d, window):
    """Both within the same bounds of the same numbers; the same bits where one
    tile takes a request's rows, whose keys the few-row kernel cuts alike.  (The
    256-row kernel weighs the blocks of trees by their rows, so that it sums a
    row's keys in other parts.)"""
    p = TreeProblem([random_tree(None, n, "chain") for n in new], [n + 333 for n in new], Hq, Hkv, d, 32, BF, window,
                    extra_cols=60)
    o, lse = _run(p)
    a = _args(p)
    o2, lse2 = fa.attention_fwd_paged(*a[:6], p.max_new, scale=p.scale, window=p.window or None)
    want = p.reference()
    check(o, lse, want, p.rows)
    check(o2, lse2, want, p.rows)
    if max(new) * Hq // Hkv <= 16:
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_rows_of_no_request_stay(cuda_lib):
    for new in ([3, 2], [60, 3]):
        r = random.Random(1)
        p = TreeProblem([random_tree(r, n, "any") for n in new], [n + 50 for n in new], 4, 2, 64, 16, BF, pad_rows=9)
        a = _args(p)
        o, lse = torch.full_like(a[0], 7.0), torch.full((4, p.total), 7.0, device="cuda")
        n = _lib.fa_fwd_paged_tree_workspace_bytes(2, p.total, p.max_new, 4, 2, 64, p.table.shape[1], 16)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        _lib.fa_fwd_paged_tree(*a, o, lse, p.max_new, p.scale, ws)
        torch.cuda.synchronize()
        assert _lib.fa_get_device_status() == _lib.FA_OK
        assert (o[p.rows:] == 7).all() and (lse[:, p.rows:] == 7).all()
        check(o, lse, p.reference(), p.rows)


@pytest.mark.parametrize("new,Hq", [([6, 5, 8], 2), ([40, 5, 64], 2), ([100, 1, 1, 1, 1], 4)])
def test_bad_parents_count_as_the_context(cuda_lib, new, Hq):
    r = random.Random(3)
    trees = [random_tree(r, n, "any") for n in new]
    trees[0][3] = trees[0][4] = -1
    p = TreeProblem(trees, [n + 70 for n in new], Hq, 1, 64, 16, HF)
    want = p.reference()
    a = _args(p)
    for row, bad in ((3, 3), (4, 1 << 30), (3, -2)):
        a[6] = p.parents.cuda()
        a[6][row] = bad
        o, lse = fa.attention_fwd_paged_tree(*a, p.max_new, scale=p.scale)
        torch.cuda.synchronize()
        assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
        check(o, lse, want, p.rows)


@pytest.mark.parametrize("new", [[6, 5, 8], [40, 5, 64]])
def test_unsound_requests_beside_sound_ones(cuda_lib, new):
    """Lengths beyond the table, offsets that decrease: reported, the others' rows are right."""
    r = random.Random(4)
    p = TreeProblem([random_tree(r, n, "any") for n in new], [n + 70 for n in new], 2, 1, 64, 16, BF)
    want = p.reference()
    a = _args(p)
    a[4] = _i32([p.lens[0], 1 << 29, p.lens[2]])
    o, lse = fa.attention_fwd_paged_tree(*a, p.max_new, scale=p.scale)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    keep = [i for i in range(p.rows) if not new[0] <= i < new[0] + new[1]]
    check(o[keep], lse[:, keep], [w[keep] if w.shape[0] == p.rows else w[:, keep] for w in want], len(keep))
    a = _args(p)
    a[3][1, 2] = p.num_pages + 3  # a page outside the pool
    o, lse = fa.attention_fwd_paged_tree(*a, p.max_new, scale=p.scale)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    check(o[keep], lse[:, keep], [w[keep] if w.shape[0] == p.rows else w[:, keep] for w in want], len(keep))


@pytest.mark.parametrize("new", [[6, 5, 8], [40, 5, 64], [100, 1, 1, 1, 1]])
def test_tree_captured_and_on_streams(cuda_lib, new):
    """Two graphs of calls with workspaces of their own, replayed at once as trees change in place."""
    r = random.Random(5)
    ps = [TreeProblem([random_tree(r, n, k) for n in new], [n + 200 for n in new], 4, 2, 64, 16, BF, seed=i, extra_cols=50)
          for i, k in enumerate(("any", "near"))]
    args = [_args(p) for p in ps]
    streams, graphs, outs = [torch.cuda.Stream() for _ in ps], [], []
    for p, a, st in zip(ps, args, streams):
        st.wait_stream(torch.cuda.current_stream())
        o, lse = fa.attention_fwd_paged_tree(*a, p.max_new, scale=p.scale, stream=st)
        st.synchronize()
        check(o, lse, p.reference(), p.rows)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(fa.attention_fwd_paged_tree(*a, p.max_new, scale=p.scale))
        graphs.append(g)
    for turn in range(3):
        for p, a in zip(ps, args):
            p.trees = [random_tree(r, n, "any") for n in new]
            a[6].copy_(_i32([x for t in p.trees for x in t]))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert _lib.fa_get_device_status() == _lib.FA_OK
        for p, (o, lse) in zip(ps, outs):
            check(o, lse, p.reference(), p.rows)


def test_workspace_bytes_and_refusals(cuda_lib):
    r = random.Random(6)
    p = TreeProblem([random_tree(r, 40, "any")], [100], 4, 2, 64, 16, BF)
    a = _args(p)
    n = _lib.fa_fwd_paged_tree_workspace_bytes(1, p.total, 40, 4, 2, 64, p.table.shape[1], 16)
    o, lse = torch.empty_like(a[0]), torch.empty(4, p.total, device="cuda")
    with pytest.raises(_lib.FAError) as e:
        _lib.fa_fwd_paged_tree(*a, o, lse, 40, p.scale, torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == _lib.FA_ERR_WORKSPACE
    _lib.fa_fwd_paged_tree(*a, o, lse, 40, p.scale, torch.empty(n, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    check(o, lse, p.reference(), p.rows)
    for bad in (a[6].long(), a[6].cpu(), a[6][:-1], torch.stack([a[6], a[6]], 1)[:, 0]):
        with pytest.raises((TypeError, ValueError)):
            fa.attention_fwd_paged_tree(*a[:6], bad, 40)
    with pytest.raises(_lib.FAError) as e:
        fa.attention_fwd_paged_tree(*a, 1025)
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED
    with pytest.raises(_lib.FAError):
        fa.attention_fwd_paged_tree(*a[:5], None, a[6], 1)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_long_context(cuda_lib, dtype):
    """More key tiles than one sum of the 256-row kernel takes, for fp16."""
    r = random.Random(7)
    p = TreeProblem([random_tree(r, 24, "any")], [40000], 2, 1, 64, 256, dtype)
    check(*_run(p), p.reference(), p.rows)


@pytest.mark.parametrize("new", [[7, 3], [60, 33]])
def test_fa_step_of_speculative_decoding(cuda_lib, new):
    """Tables, append, tree attention, the accepted path moved, the rest given
    back; the next step's rows then see the same keys as a cache that was
    written in order."""
    r = random.Random(8)
    Hq, Hkv, d, ps, num, width = 4, 2, 64, 16, 64, 20
    g = torch.Generator("cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)

    k_cache, v_cache = rand(num, Hkv, ps, d), rand(num, Hkv, ps, d)
    table, free = _i32([-1] * 2 * width).view(2, width), _i32(r.sample(range(num), num))
    lens, cu, slots, counts = fa.paged_tables(_i32([0, 0]), _i32([75, 33]), table, free, ps, num, 108)
    k, v = rand(108, Hkv, d), rand(108, Hkv, d)
    fa.paged_append(k, v, slots, k_cache, v_cache)
    ks, vs = [k[:75], k[75:]], [v[:75], v[75:]]
    trees = [random_tree(r, n, "any") for n in new]
    total = sum(new)
    base = lens
    lens, cu, slots, counts = fa.paged_tables(base, _i32(new), table, free, ps, num, total, free_start=counts[:1].clone())
    k, v, q = rand(total, Hkv, d), rand(total, Hkv, d), rand(total, Hq, d)
    fa.paged_append(k, v, slots, k_cache, v_cache)
    o, lse = fa.attention_fwd_paged_tree(q, k_cache, v_cache, table, lens, cu, _i32([x for t in trees for x in t]),
                                         max(new))
    # every row as if its path alone had been appended to a cache of its own
    row = 0
    for b, n in enumerate(new):
        for i in range(n):
            path, j = [], i
            while j >= 0:
                path.insert(0, row - i + j)
                j = trees[b][j]
            kk, vv = torch.cat([ks[b], k[path]]), torch.cat([vs[b], v[path]])
            pages = -(-len(kk) // ps)
            own = [torch.zeros(pages, ps, Hkv, d, dtype=BF, device="cuda") for _ in range(2)]
            for c, x in zip(own, (kk, vv)):
                c.view(-1, Hkv, d)[: len(x)] = x
            own = [c.transpose(1, 2).contiguous() for c in own]
            o2, lse2 = fa.attention_fwd_paged(q[row:row + 1], *own, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                                              _i32([len(kk)]))
            # both are within a few roundings (2^-8 of values below 4) of the same number
            assert (o[row] - o2[0]).abs().max() <= 2 * 2.0 ** -8 * 4 and (lse[:, row] - lse2[:, 0]).abs().max() < 1e-4
            row += 1
    # the longest path is accepted
    best = [max(range(n), key=lambda i: len(path_of(t, i))) for n, t in zip(new, trees)]
    keep = [path_of(t, i)[::-1] for t, i in zip(trees, best)]
    most = max(map(len, keep))
    fa.paged_compact(torch.stack([_i32(p + [0] * (most - len(p))) for p in keep]), _i32(map(len, keep)), base, table,
                     k_cache, v_cache)
    after = base + _i32(map(len, keep))
    counts = fa.paged_free(lens, after, table, free, counts[:1].clone(), ps, num)
    row = 0
    for b, n in enumerate(new):
        ks[b], vs[b] = (torch.cat([x, y[[row + j for j in keep[b]]]]) for x, y in ((ks[b], k), (vs[b], v)))
        row += n
        for t in range(int(after[b])):
            assert torch.equal(k_cache[table[b, t // ps], :, t % ps], ks[b][t])
            assert torch.equal(v_cache[table[b, t // ps], :, t % ps], vs[b][t])
    used = sum(-(-n // ps) for n in after.tolist())
    assert counts.tolist() == [used, 0]
    held = [int(table[b, c]) for b in range(2) for c in range(-(-int(after[b]) // ps))]
    assert sorted(held + free[used:].tolist()) == list(range(num))
    assert _lib.fa_get_device_status() == _lib.FA_OK
