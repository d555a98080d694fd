"""The paged-cache operators against plain forms in 64 bits (bounds: _paged)."""
import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import Problem, check, pages_of, tables_reference

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _call(p, single=False, **kw):
    args = [p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda()]
    fn = fa.attention_fwd_paged
    if p.prefix:
        fn = fa.attention_fwd_paged_prefix
        args += [_i32(p.front), p.prefix]
    args += [p.table.cuda(), _i32(p.lens)]
    if not single:
        kw = {"cu_seqlens": p.cu.cuda(), "max_new": p.max_new, **kw}
    return fn(*args, scale=p.scale, window=p.window or None, **kw)


def _run(p, single=False, **kw):
    o, lse = _call(p, single, **kw)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    return o, lse


# lens, new, Hq, Hkv, d, page_size, dtype, window, prefix
ATTENTION = [
    # one token a request: lengths around tiles and pages
    ([1], [1], 1, 1, 128, 16, BF, 0, 0),
    ([1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300], [1] * 12, 4, 4, 128, 16, BF, 0, 0),
    ([255, 256, 257, 1000], [1] * 4, 8, 2, 128, 64, HF, 0, 0),
    ([511, 7, 640], [1] * 3, 6, 2, 64, 32, BF, 0, 0),
    ([33, 1500], [1, 1], 16, 1, 64, 256, HF, 0, 0),
    ([700, 31], [1, 1], 20, 1, 128, 128, BF, 0, 0),     # more heads than one 16-row tile
    ([90, 400], [1, 1], 40, 1, 64, 64, HF, 0, 0),
    # no keys, no rows, a row that sees nothing, more rows than keys
    ([0, 5, 0, 9], [1, 1, 0, 0], 4, 2, 128, 16, BF, 0, 0),
    ([3, 0, 40], [5, 2, 1], 4, 2, 64, 16, HF, 0, 0),
    ([2], [300], 2, 1, 128, 32, BF, 0, 0),
    # a few rows a request
    ([100, 17, 4, 333], [3, 1, 4, 2], 8, 2, 128, 16, BF, 0, 0),
    ([1000, 64], [8, 5], 4, 2, 64, 64, HF, 0, 0),
    # chunks of a prompt, alone and among single tokens
    ([300], [300], 4, 2, 128, 64, BF, 0, 0),
    ([257, 1000, 5], [257, 130, 1], 3, 1, 64, 16, HF, 0, 0),
    ([640, 900, 33, 128], [1, 513, 1, 128], 8, 1, 128, 32, BF, 0, 0),
    ([400, 129], [70, 129], 5, 1, 128, 128, HF, 0, 0),
    # up to 128 rows a block, by turns with more: one, two, three and more tiles
    ([100, 130, 300, 1000, 513], [7, 20, 5, 30, 9], 4, 1, 128, 64, BF, 0, 0),
    ([200, 1000, 700, 60, 900], [5, 200, 6, 3, 40], 4, 1, 64, 16, HF, 0, 0),
    ([1500, 900, 260, 1400], [9, 100, 130, 20], 8, 2, 128, 128, BF, 0, 0),
    ([1300, 700, 900], [20, 6, 31], 4, 1, 128, 32, HF, 300, 0),
    # one long chunk among many short requests: both kernels at once
    ([400, 90, 1, 700, 64, 0, 129, 1500, 33], [300, 1, 1, 2, 1, 0, 1, 1, 3], 8, 2, 128, 16, BF, 0, 0),
    ([900, 10, 2000, 77, 65, 300, 8, 1], [260, 4, 1, 5, 1, 2, 8, 1], 4, 2, 64, 64, HF, 0, 0),
    ([500, 3, 130, 1000, 17, 260, 64, 9, 512, 70], [200, 3, 1, 1, 1, 20, 2, 1, 1, 9], 16, 2, 128, 32, HF, 200, 0),
    ([200, 1, 40, 300, 5, 64, 128, 2], [150, 1, 4, 1, 1, 1, 2, 1], 8, 2, 64, 16, BF, 0, 333),
    ([260, 7, 90, 30, 400, 1, 1, 19], [129, 1, 1, 1, 3, 1, 1, 1], 4, 1, 128, 128, BF, 100, 150),
    # sliding windows
    ([500, 20, 129], [1] * 3, 4, 2, 128, 16, BF, 100, 0),
    ([500, 20, 129], [1] * 3, 4, 2, 64, 64, HF, 1, 0),
    ([900, 300], [200, 7], 4, 1, 128, 32, BF, 64, 0),
    ([900, 300, 1], [6, 7, 1], 2, 1, 64, 16, HF, 130, 0),
    # a shared prefix
    ([1, 17, 40], [1] * 3, 4, 2, 128, 16, BF, 0, 100),
    ([5, 200, 64, 1], [1] * 4, 8, 1, 64, 64, HF, 0, 1),
    ([30, 9], [1, 1], 16, 2, 128, 128, BF, 0, 700),
    ([50, 3, 130], [4, 3, 130], 4, 2, 128, 32, HF, 0, 257),
    ([0, 0, 7], [1, 0, 1], 4, 2, 64, 16, BF, 0, 33),     # nothing but the prefix
    ([1, 2], [5, 2], 2, 2, 64, 16, HF, 0, 3),           # rows inside and before the prefix
    ([80, 10, 300], [1] * 3, 4, 2, 128, 16, BF, 90, 200),  # windows that end in the prefix, and behind it
    ([80, 10, 300], [20, 10, 200], 4, 2, 64, 64, HF, 50, 129),
    ([12] * 70, [1] * 70, 8, 1, 128, 16, BF, 0, 515),   # more rows of one head than one tile
    # enough requests, on a long enough prefix, that it gets a pass of its own
    ([1 + (7 * i) % 90 for i in range(70)], [1] * 70, 8, 2, 128, 64, BF, 0, 2100),
    ([3 + (5 * i) % 50 for i in range(140)], [1 + i % 3 for i in range(140)], 8, 4, 64, 16, HF, 0, 1001),
    ([2 * (i % 40) for i in range(90)], [1] * 90, 4, 4, 128, 32, BF, 0, 700),       # some without keys of their own
    ([4 + (11 * i) % 300 for i in range(80)], [1 + i % 4 for i in range(80)], 4, 4, 64, 128, BF, 260, 1200),
    ([4 + (11 * i) % 300 for i in range(80)], [1 + i % 2 for i in range(80)], 16, 2, 128, 16, HF, 700, 1500),
]


@pytest.mark.parametrize("lens,new,Hq,Hkv,d,ps,dtype,window,prefix", ATTENTION)
@pytest.mark.parametrize("cols", [1, 80])  # a wide table may hold long sequences: their keys are split
def test_attention_matches_64_bits(cuda_lib, lens, new, Hq, Hkv, d, ps, dtype, window, prefix, cols):
    p = Problem(lens, new, Hq, Hkv, d, ps, dtype, window, prefix, seed=d + ps, extra_cols=cols)
    want = p.reference()
    check(*_run(p), want, p.rows)
    if all(n == 1 for n in new):  # the same without offsets
        check(*_run(p, single=True), want, p.rows)


@pytest.mark.parametrize("seed", range(24))
def test_attention_random(cuda_lib, seed):
    import random
    r = random.Random(seed)
    Hkv, group, d = r.choice([1, 2, 3, 4]), r.choice([1, 2, 3, 5, 7, 8, 16, 24]), r.choice([64, 128])
    B = r.choice([1, 2, 5, 9])
    most = r.choice([1, 1, 4, 40, 200])
    new = [r.randint(0, most) for _ in range(B)]
    new[r.randrange(B)] = most
    lens = [n + r.choice([0, 0, r.randint(0, 60), r.randint(0, 700)]) for n in new]
    window = r.choice([0, 0, r.randint(1, 300)])
    prefix = r.choice([0, 0, r.randint(1, 400)])
    p = Problem(lens, new, Hkv * group, Hkv, d, r.choice([16, 32, 64, 128, 256]), r.choice([BF, HF]), window, prefix,
                seed=seed, pad_rows=r.choice([0, 3]), sharp=r.choice([1.0, 4.0]), extra_cols=r.choice([1, 100]))
    # a bound on the rows that no request reaches is as good
    check(*_run(p, max_new=p.max_new + r.choice([0, 0, 50])), p.reference(), p.rows)


@pytest.mark.parametrize("lens,new,Hq,Hkv,d,ps,prefix", [
    ([3 + (7 * i) % 90 for i in range(700)], [1] * 700, 4, 2, 64, 16, 0),
    ([3 + (7 * i) % 90 for i in range(700)], [1] * 700, 4, 1, 64, 32, 70),
    ([20 + (11 * i) % 150 for i in range(300)], [1 + (5 * i) % 19 for i in range(300)], 8, 1, 64, 16, 0),
    ([20 + (11 * i) % 150 for i in range(300)], [1 + (5 * i) % 19 for i in range(300)], 4, 1, 128, 16, 40),
    ([300, 5], [2, 2], 128, 1, 64, 64, 0),       # a token fills a tile
    ([300, 5], [3, 1], 200, 1, 64, 64, 20),      # and does not divide one
    ([200], [3], 300, 1, 128, 32, 0),            # a token is more than a block
    ([2500], [2300], 2, 1, 64, 16, 0),           # many blocks of one request
    ([30 + (13 * i) % 400 for i in range(400)] + [900], [1 + (3 * i) % 4 for i in range(400)] + [800], 4, 1, 64, 16, 0),
    ([30 + (13 * i) % 400 for i in range(300)] + [900], [1] * 300 + [500], 8, 2, 128, 32, 60),
])
def test_many_requests_and_wide_groups(cuda_lib, lens, new, Hq, Hkv, d, ps, prefix):
    p = Problem(lens, new, Hq, Hkv, d, ps, BF, 0, prefix, extra_cols=70)
    check(*_run(p), p.reference(), p.rows)


@pytest.mark.parametrize("lens,new,Hq,Hkv,d,ps,dtype,window,prefix", [
    # the prefix read with each request's own keys: around tiles and pages of it
    ([70, 200, 130], [70, 200, 130], 4, 2, 128, 64, BF, 0, 1000),
    ([100, 300, 40], [33, 120, 40], 3, 1, 64, 256, HF, 0, 129),
    ([200, 500], [200, 150], 8, 1, 64, 16, BF, 0, 128),
    ([300, 90], [290, 80], 4, 1, 128, 32, HF, 0, 1),
    ([3000], [200], 3, 1, 128, 128, BF, 0, 5000),          # divided among CTAs, also within the prefix
    ([5, 0, 300], [100, 40, 300], 4, 2, 64, 16, BF, 0, 77),  # rows inside the prefix, and before it
    ([0, 0], [300, 150], 2, 2, 128, 64, HF, 0, 700),
    ([900, 3, 40, 1, 0, 6], [300, 1, 1, 1, 0, 2], 8, 2, 128, 16, BF, 0, 400),  # by both kernels
    # windows that end in the prefix, behind it, and, block by block, both
    ([70, 200, 130], [70, 200, 130], 4, 2, 64, 16, HF, 500, 1000),
    ([1500], [1500], 2, 1, 128, 64, BF, 200, 500),
    ([1200, 5], [700, 5], 4, 1, 64, 32, BF, 600, 333),
    ([900, 3, 40, 1, 0, 6], [300, 1, 1, 1, 0, 2], 8, 2, 64, 64, HF, 350, 400),
    # a pass of its own over the prefix, before the 256-row kernel's and beside both
    ([20 + 5 * i for i in range(12)], [9 + i for i in range(12)], 4, 4, 64, 32, BF, 0, 6000),
    ([20 + 5 * i for i in range(12)], [9 + i for i in range(12)], 12, 4, 128, 16, HF, 4000, 6000),
    ([150] + [20 + i for i in range(30)], [100] + [1] * 30, 8, 2, 128, 64, BF, 0, 6000),
    ([150] + [20 + i for i in range(30)], [100] + [1 + i % 3 for i in range(30)], 4, 2, 64, 16, HF, 1000, 9000),
])
def test_prefix_of_many_rows(cuda_lib, lens, new, Hq, Hkv, d, ps, dtype, window, prefix):
    p = Problem(lens, new, Hq, Hkv, d, ps, dtype, window, prefix, seed=3, pad_rows=2, extra_cols=40)
    check(*_run(p), p.reference(), p.rows)


def test_long_sequence_among_short_ones(cuda_lib):
    """One request far longer than the others: its keys are split over many
    blocks and merged, theirs are not."""
    p = Problem([20000, 1, 130, 64], [1] * 4, 8, 2, 128, 64, BF, seed=3)
    check(*_run(p, single=True), p.reference(), p.rows)


def test_equal_calls_give_equal_bits(cuda_lib):
    for case in (([3000, 700, 1], [1] * 3, 8, 2, 128, 64, BF, 0, 500), ([800, 300], [300, 70], 4, 1, 64, 16, HF, 0, 0),
                 ([30, 9] * 40, [1] * 80, 8, 2, 128, 16, BF, 0, 2000), ([800, 30, 900] * 4, [250, 1, 1] + [1] * 9, 8, 2,
                                                                       128, 64, BF, 0, 0)):
        p = Problem(*case)
        a, b = _run(p), _run(p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("new,prefix", [([1, 1], 0), ([40, 300], 0), ([1, 1], 90), ([200, 1], 90)])
@pytest.mark.parametrize("window", [1000, 2 ** 31 - 1])
def test_window_of_all_keys_is_none(cuda_lib, new, prefix, window):
    p = Problem([300, 310], new, 4, 2, 64, 16, BF, 0, prefix)
    a = _run(p)
    p.window = window
    b = _run(p)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pages_in_several_places(cuda_lib):
    """Requests may share pages, and a table name a page twice."""
    p = Problem([64, 64], [1, 1], 4, 2, 64, 16, BF)
    table = p.table[:1, [0, 1, 0, 1, 0]].repeat(2, 1).contiguous()
    q = p.q[:1].repeat(2, 1, 1).contiguous().cuda()
    o, lse = fa.attention_fwd_paged(q, p.k_cache.cuda(), p.v_cache.cuda(), table.cuda(), _i32([64, 64]), scale=p.scale)
    p.k[0] = torch.cat([p.k[0][:, :32]] * 2, 1)
    p.v[0] = torch.cat([p.v[0][:, :32]] * 2, 1)
    p.lens, p.new, p.rows = p.lens[:1], [1], 1
    check(o[:1], lse[:, :1], p.reference(), 1)
    assert torch.equal(o[0], o[1]) and torch.equal(lse[:, 0], lse[:, 1])


def test_prefix_equals_the_same_keys_unshared(cuda_lib):
    """Both calls stay within their bounds of the same 64-bit result."""
    p = Problem([70, 5, 129], [1, 1, 1], 8, 2, 128, 16, BF, 0, 160, seed=5)
    want = p.reference()
    check(*_run(p), want, p.rows)
    table = p.table.clone()
    wide = torch.full((3, table.shape[1] + 10), -1, dtype=torch.int32)
    wide[:, :10] = torch.tensor(p.front, dtype=torch.int32)
    wide[:, 10:] = table
    o, lse = fa.attention_fwd_paged(p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), wide.cuda(),
                                    _i32(n + 160 for n in p.lens), scale=p.scale)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    check(o, lse, want, p.rows)


@pytest.mark.parametrize("new,prefix", [([1, 1], 0), ([40, 3], 0), ([1, 1], 50), ([40, 3], 50), ([1, 1], 20000)])
def test_rows_of_no_request_stay_as_they_are(cuda_lib, new, prefix):
    p = Problem([200, 64], new, 4, 2, 128, 16, BF, 0, prefix, pad_rows=37)
    o = torch.full_like(p.q, 7.0).cuda()
    lse = torch.full((4, p.total), 7.0, device="cuda")
    ws = torch.full((_lib.fa_fwd_paged_workspace_bytes(2, p.total, p.max_new, 4, 2, 128, p.table.shape[1], 16,
                                                       prefix),), 0xFF, dtype=torch.uint8, device="cuda")
    args = [p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda()]
    tail = (p.table.cuda(), _i32(p.lens), p.cu.cuda(), o, lse, p.max_new, p.scale, ws)
    if prefix:
        _lib.fa_fwd_paged_prefix(*args, _i32(p.front), prefix, *tail)
    else:
        _lib.fa_fwd_paged(*args, *tail)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    check(o, lse, p.reference(), p.rows)
    assert (o[p.rows:] == 7.0).all() and (lse[:, p.rows:] == 7.0).all()


@pytest.mark.parametrize("new", [[1, 1, 1], [30, 1, 70], [2, 1, 190]])
@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "offsets", "too many rows"])
def test_bad_device_values_are_reported(cuda_lib, what, new, prefix):
    """Values read on the device that would lead out of range are refused
    there: the call returns, the status says so, and the other requests'
    rows are right."""
    p = Problem([150, 90, 200], new, 4, 2, 64, 16, BF, 0, prefix)
    want = p.reference()
    lens, cu, table, most = list(p.lens), p.cu.clone(), p.table.clone(), p.max_new
    if what == "page":
        table[1, 0] = p.num_pages
    elif what == "negative page":
        table[1, 2] = -1
    elif what == "length":
        lens[1] = p.table.shape[1] * 16 + 1
    elif what == "negative length":
        lens[1] = -1
    elif what == "offsets":
        cu[3] = p.total + 1
    else:
        if p.max_new == 1:
            pytest.skip("one row is the least bound")
        most = 60
    tail = (table.cuda(), _i32(lens), cu.cuda(), most)
    args = (p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda())
    if prefix:
        o, lse = fa.attention_fwd_paged_prefix(*args, _i32(p.front), prefix, *tail, scale=p.scale)
    else:
        o, lse = fa.attention_fwd_paged(*args, *tail, scale=p.scale)
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    n = new[0]  # the first request is sound in every case
    check(o, lse, (want[0][:n], want[1][:, :n], want[2][:n], want[3][:, :n]), n)
    assert _lib.fa_get_device_status() == _lib.FA_OK


@pytest.mark.parametrize("new,prefix", [([1, 1, 1], 0), ([1, 1, 1], 40), ([1, 1, 1], 80000), ([2, 1, 190], 0),
                                        ([2, 1, 190], 40), ([90, 70, 80], 0), ([90, 70, 80], 2000)])
@pytest.mark.parametrize("at,value", [(0, -3), (0, 2 ** 30), (3, -1), (3, 0), (3, 2 ** 31 - 1)])
def test_bad_outer_offsets_concern_their_request(cuda_lib, at, value, new, prefix):
    """The first or the last offset bounds the rows of all requests: a wrong
    one must not cut off those of the others."""
    p = Problem([150, 90, 200], new, 4, 2, 64, 16, BF, 0, prefix, extra_cols=80)
    want, cu = p.reference(), p.cu.clone()
    cu[at] = value
    tail = (p.table.cuda(), _i32(p.lens), cu.cuda(), p.max_new)
    args = (p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda())
    if prefix:
        o, lse = fa.attention_fwd_paged_prefix(*args, _i32(p.front), prefix, *tail, scale=p.scale)
    else:
        o, lse = fa.attention_fwd_paged(*args, *tail, scale=p.scale)
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    lo, hi = (int(p.cu[1]), p.rows) if at == 0 else (0, int(p.cu[2]))
    check(o[lo:hi], lse[:, lo:hi], (want[0][lo:hi], want[1][:, lo:hi], want[2][lo:hi], want[3][:, lo:hi]), hi - lo)
    assert _lib.fa_get_device_status() == _lib.FA_OK


@pytest.mark.parametrize("lens,new,prefix", [([150, 90, 200], [1, 1, 1], 40), ([150, 90, 200], [1, 1, 1], 80000),
                                             ([150, 90, 200], [90, 70, 80], 2000), ([30] * 12, [20] * 12, 6000)])
@pytest.mark.parametrize("page", [-1, 10 ** 6, 2 ** 31 - 1])
def test_bad_prefix_pages_are_reported(cuda_lib, lens, new, prefix, page):
    p = Problem(lens, new, 4, 2, 64, 16, BF, 0, prefix, extra_cols=80)
    good = list(p.front)
    p.front[len(good) // 2] = page
    _call(p)
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    p.front = good
    check(*_run(p), p.reference(), p.rows)


# --------------------------------------------------------------- tables


def _tables_case(cached, new, page_size, free, start=0, cols=None, total=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    cols = cols or max(pages_of(c + n, page_size) for c, n in zip(cached, new)) + 1
    total = total or max(1, sum(new))
    num_pages = sum(pages_of(c, page_size) for c in cached) + free + 5
    ids = torch.randperm(num_pages, generator=g).tolist()
    table = torch.full((len(cached), cols), -1, dtype=torch.int32)
    for b, c in enumerate(cached):
        for i in range(pages_of(c, page_size)):
            table[b, i] = ids.pop()
    pool = [ids.pop() for _ in range(free)]
    want = tables_reference(cached, new, table, pool, start, page_size, total)
    dev = table.cuda()
    got = fa.paged_tables(_i32(cached), _i32(new), dev, _i32(pool), page_size, num_pages, total,
                          free_start=_i32([start]) if start else None)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    assert torch.equal(dev.cpu(), want[0])
    for g_, w in zip(got, want[1:]):
        assert g_.tolist() == w


@pytest.mark.parametrize("cached,new,page_size,free,start,total", [
    ([0], [1], 16, 1, 0, 1),
    ([15, 16, 17, 0], [1, 1, 1, 0], 16, 4, 0, 3),
    ([0, 0, 0], [0, 0, 0], 64, 0, 0, 1),                  # nothing to do
    ([5, 6], [1, 1], 32, 0, 0, 9),                        # no page needed, none there, padded rows
    ([0, 100, 33], [200, 1, 70], 16, 40, 7, 300),
    ([0, 0, 3], [100, 64, 5], 16, 7, 0, 169),             # exactly seven for the first, none for the second
    ([0, 0, 3], [100, 64, 5], 16, 6, 0, 169),             # the first is not served, nor the second
    ([1, 2, 3], [300, 0, 17], 256, 1, 1, 320),            # the pool is empty from its start on
])
def test_tables(cuda_lib, cached, new, page_size, free, start, total):
    _tables_case(cached, new, page_size, free, start, total=total)


@pytest.mark.parametrize("seed", range(6))
def test_tables_random(cuda_lib, seed):
    import random
    r = random.Random(seed)
    B = r.choice([1, 33, 255, 256, 257, 1500])
    ps = r.choice([16, 32, 64, 128, 256])
    cached = [r.choice([0, r.randint(0, 400)]) for _ in range(B)]
    new = [r.choice([0, 1, 1, r.randint(0, 100)]) for _ in range(B)]
    need = sum(pages_of(c + n, ps) - pages_of(c, ps) for c, n in zip(cached, new))
    _tables_case(cached, new, ps, r.choice([need, need + 3, need // 2]), total=sum(new) + r.choice([1, 50]), seed=seed)


@pytest.mark.parametrize("cached,new,page_size,free,total", [
    ([10, 0, 5], [10, 17, 1], 16, 2, 30),                          # the last needs no page, the one before gets none
    ([3] * 400, [200 + i % 7 for i in range(400)], 16, 5200, 81203),  # four rows a thread, the last one's fewer
    ([3] * 400, [200 + i % 7 for i in range(400)], 16, 3000, 81203),  # and a pool that runs out on the way
    ([7], [200000], 16, 12600, 200001),                            # one prompt of many pages
    ([16 * (i % 9) + 15 for i in range(1024)], [i % 3 for i in range(1024)], 16, 300, 1100),
])
def test_tables_over_the_whole_grid(cuda_lib, cached, new, page_size, free, total):
    _tables_case(cached, new, page_size, free, total=total)


def test_tables_most_requests(cuda_lib):
    B = 16384
    _tables_case([i % 40 for i in range(B)], [(7 * i) % 5 for i in range(B)], 16, B)


@pytest.mark.parametrize("what", ["cached", "new", "sum", "rows", "start", "free page", "held page"])
def test_tables_bad_values_are_reported(cuda_lib, what):
    table = torch.tensor([[3, 0, 0], [5, 0, 0]], dtype=torch.int32)
    cached, new, pool, start, total = [10, 4], [1, 20], [7, 8], 0, 21
    if what == "cached":
        cached[1] = -4
    elif what == "new":
        new[1] = -1
    elif what == "sum":
        new[1] = 45
    elif what == "rows":
        total = 5
    elif what == "start":
        start = 3
    elif what == "free page":
        pool[0] = 99
    else:
        table[1, 0] = -3
    slots = fa.paged_tables(_i32(cached), _i32(new), table.cuda(), _i32(pool), 16, 12, total,
                            free_start=_i32([start]))[2]
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    assert slots[0].item() == 3 * 16 + 10
    assert ((slots >= -1) & (slots < 12 * 16)).all()


# --------------------------------------------------------------- append


@pytest.mark.parametrize("total,Hkv,d,ps,dtype", [
    (1, 1, 64, 16, BF), (3, 2, 128, 16, HF), (257, 8, 128, 64, BF), (100, 3, 64, 256, HF), (9, 40, 128, 32, BF)])
def test_append_writes_named_slots_only(cuda_lib, total, Hkv, d, ps, dtype):
    g = torch.Generator().manual_seed(total)
    pages = pages_of(total, ps) + 2
    kc, vc = (torch.randn(pages, Hkv, ps, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(total, Hkv, d, generator=g).to(dtype) for _ in range(2))
    slots = torch.randperm(pages * ps, generator=g)[:total].to(torch.int32)
    slots[::5] = -1
    want = [kc.clone(), vc.clone()]
    for r, s in enumerate(slots.tolist()):
        if s >= 0:
            want[0][s // ps, :, s % ps], want[1][s // ps, :, s % ps] = k[r], v[r]
    kc, vc = kc.cuda(), vc.cuda()
    fa.paged_append(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


def test_append_reports_slots_behind_the_cache(cuda_lib):
    kc, vc = (torch.zeros(2, 1, 16, 64, dtype=BF, device="cuda") for _ in range(2))
    k = torch.ones(3, 1, 64, dtype=BF, device="cuda")
    fa.paged_append(k, k, _i32([5, 32, 2 ** 31 - 1]), kc, vc)
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    assert kc.sum().item() == 64 and kc[0, 0, 5].sum().item() == 64


# ------------------------------------------------ the operators together


@pytest.mark.parametrize("Hq,Hkv,d,ps,dtype,window", [(4, 2, 128, 16, BF, None), (6, 1, 64, 64, HF, 50)])
def test_serving_run(cuda_lib, Hq, Hkv, d, ps, dtype, window):
    """Prompts in chunks, then single tokens: at every step tables, append and
    attention, against the packed forward over the whole sequences."""
    g = torch.Generator().manual_seed(d)
    final = [90, 33, 201]
    B = len(final)
    x = {n: [torch.randn(f, h, d, generator=g).to(dtype).cuda() for f in final]
         for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    cu = _i32([0, 90, 123, 324])
    whole, whole_lse = fa.attention_fwd_varlen(*(torch.cat(x[n]) for n in "qkv"), cu, causal=True, window=window)
    whole, whole_lse = whole.split(final), whole_lse.split(final, 1)
    pages = sum(pages_of(f, ps) for f in final) + 2
    kc, vc = (torch.full((pages, Hkv, ps, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    table = torch.full((B, pages_of(max(final), ps)), -1, dtype=torch.int32, device="cuda")
    pool = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    lens, start, done = _i32([0] * B), None, [0] * B
    for step in range(200):
        new = [min(f - n, 64 if n + 64 <= f - 20 else 1) for f, n in zip(final, done)]
        if not any(new):
            break
        total = sum(new) + (step % 3)  # some steps are padded
        lens, cu, slots, counts = fa.paged_tables(lens, _i32(new), table, pool, ps, pages, total, free_start=start)
        start = counts[:1].clone()
        rows = {n: torch.cat([t[a:a + m] for t, a, m in zip(x[n], done, new)]) for n in "qkv"}
        pad = total - sum(new)
        if pad:
            rows = {n: torch.cat([t, t.new_full((pad,) + t.shape[1:], float("nan"))]) for n, t in rows.items()}
        fa.paged_append(rows["k"], rows["v"], slots, kc, vc)
        o, lse = fa.attention_fwd_paged(rows["q"], kc, vc, table, lens, cu, max(new), window=window)
        r = 0
        for b, m in enumerate(new):
            part = slice(done[b], done[b] + m)
            # both sides round P and O to the 16-bit type: 2 u each of values up to max |V| < 6
            tol = 4 * torch.finfo(dtype).eps / 2 * 6
            assert (o[r:r + m].float() - whole[b][part].float()).abs().max() <= tol if m else True
            if m:
                assert (lse[:, r:r + m] - whole_lse[b][:, part]).abs().max() <= 1e-4
            r += m
            done[b] += m
    assert done == final
    assert _lib.fa_get_device_status() == _lib.FA_OK


def test_captured_step_follows_its_inputs(cuda_lib):
    """tables, append and attention in one graph, replayed with other lengths
    and values in the same tensors."""
    ps, Hq, Hkv, d, B, pages = 16, 4, 2, 64, 3, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    kc, vc = (torch.randn(pages, Hkv, ps, d, generator=g, device="cuda").to(BF) for _ in range(2))
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table0 = ids[:30].reshape(3, 10).contiguous()
    table, pool = table0.clone(), ids[30:].contiguous()
    lens, new = _i32([40, 7, 100]), _i32([1, 1, 1])
    q, k, v = (torch.randn(B, h, d, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))

    def step():
        seq, cu, slots, _ = fa.paged_tables(lens, new, table, pool, ps, pages, B)
        fa.paged_append(k, v, slots, kc, vc)
        return fa.attention_fwd_paged(q, kc, vc, table, seq)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for now in ([40, 7, 100], [16, 0, 143], [1, 90, 31]):
        lens.copy_(_i32(now))
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
        table.copy_(table0)
        kc0, vc0 = kc.clone(), vc.clone()
        graph.replay()
        got = o.clone(), lse.clone()
        table.copy_(table0)
        kc.copy_(kc0)
        vc.copy_(vc0)
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert _lib.fa_get_device_status() == _lib.FA_OK


@pytest.mark.parametrize("new,prefix", [([70, 200, 130], 0), ([300, 1, 1, 2, 1, 1], 0), ([1, 1, 1], 200),
                                        ([300, 1, 1, 2, 1, 1], 200), ([1, 2] * 40, 2000)])
def test_captured_forward_of_every_kernel(cuda_lib, new, prefix):
    """Captured with one problem's values, replayed with another's of the same
    shapes, and next to a graph of the other kernels."""
    ps = [Problem([n + 37 * (i % 8) + 90 for i, n in enumerate(new)], new, 8, 2, 128, 16, BF, 0, prefix, seed=s)
          for s in (1, 2)]
    names = ("q", "k_cache", "v_cache", "table", "cu")
    dev = {n: getattr(ps[0], n).cuda() for n in names}
    dev["lens"], dev["front"] = _i32(ps[0].lens), _i32(ps[0].front or [0])

    def call():
        args = (dev["q"], dev["k_cache"], dev["v_cache"])
        tail = (dev["table"], dev["lens"], dev["cu"], max(new))
        if prefix:
            return fa.attention_fwd_paged_prefix(*args, dev["front"], prefix, *tail)
        return fa.attention_fwd_paged(*args, *tail)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = call()
        o, lse = call()
    for p in (ps[1], ps[0]):
        for n in names:
            dev[n].copy_(getattr(p, n))
        dev["lens"].copy_(_i32(p.lens))
        dev["front"].copy_(_i32(p.front or [0]))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        check(o, lse, p.reference(), p.rows)
        assert torch.equal(first[0], o) and torch.equal(first[1], lse)
    assert _lib.fa_get_device_status() == _lib.FA_OK


def test_two_streams_at_once(cuda_lib):
    """Two calls in flight on streams of their own (outputs and workspace are
    allocated on the stream that is named)."""
    ps = [Problem([90, 12, 77] * 20, [1] * 60, 8, 2, 128, 64, BF, 0, 2200, seed=1),
          Problem([500, 333], [64, 200], 4, 1, 64, 16, HF, 0, 0, seed=2)]
    want = [p.reference() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    data = []
    for p in ps:
        args = [p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda()]
        if p.prefix:
            args += [_i32(p.front), p.prefix]
        data.append(args + [p.table.cuda(), _i32(p.lens), p.cu.cuda(), p.max_new])
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for p, s, args in zip(ps, streams, data):
            fn = fa.attention_fwd_paged_prefix if p.prefix else fa.attention_fwd_paged
            got.append(fn(*args, scale=p.scale, stream=s))
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    for i, (o, lse) in enumerate(got):
        check(o, lse, want[i % 2], ps[i % 2].rows)


def test_python_layer_refuses(cuda_lib):
    p = Problem([50, 20], [1, 1], 4, 2, 64, 16, BF)
    q, kc, vc, table, lens = p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), p.table.cuda(), _i32(p.lens)
    call = fa.attention_fwd_paged
    for bad in [(q, kc.half(), vc, table, lens), (q.float(), kc, vc, table, lens), (q, kc, vc, table.long(), lens)]:
        with pytest.raises(TypeError):
            call(*bad)
    for bad in [(q, kc.transpose(2, 3), vc, table, lens), (q, kc, vc[1:], table, lens), (q, kc, vc, table, lens[:1]),
                (q, kc, vc, table.t(), lens), (q, kc, vc, table.cpu(), lens), (q[..., :32], kc, vc, table, lens),
                (q[:, ::2], kc, vc, table, lens)]:
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(ValueError):
        call(q, kc, vc, table, lens, window=0)
    with pytest.raises(ValueError):  # two pages of 16 hold no 33 tokens
        fa.attention_fwd_paged_prefix(q, kc, vc, _i32([0, 1]), 33, table, lens)
    with pytest.raises(_lib.FAError):
        call(q[:1].contiguous(), kc, vc, table, lens)
    with pytest.raises(TypeError):
        fa.paged_append(q[:, :2].contiguous().half(), q[:, :2].contiguous(), lens, kc, vc)
    with pytest.raises(ValueError):
        fa.paged_append(q[:, :1].contiguous(), q[:, :1].contiguous(), lens, kc, vc)
    with pytest.raises(ValueError):
        fa.paged_tables(lens, lens[:1], table, lens, 16, p.num_pages, 2)


def test_python_layer_refuses_numbers_past_32_bits(cuda_lib):
    """The low 32 bits of a number would be another one."""
    p = Problem([50, 20], [1, 1], 4, 2, 64, 16, BF)
    args = p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda()
    table, lens, pages = p.table.cuda(), _i32(p.lens), _i32([0])
    for window, most in [(2 ** 32 + 1, 1), (None, 2 ** 32 + 1)]:
        with pytest.raises(ValueError):
            fa.attention_fwd_paged(*args, table, lens, p.cu.cuda(), most, window=window)
        with pytest.raises(ValueError):
            fa.attention_fwd_paged_prefix(*args, pages, 16, table, lens, p.cu.cuda(), most, window=window)
    with pytest.raises(ValueError):
        fa.attention_fwd_paged_prefix(*args, pages, 16 - 2 ** 32, table, lens)
    for page_size, num_pages in [(2 ** 32 + 16, p.num_pages), (16, 2 ** 32 + p.num_pages)]:
        with pytest.raises(ValueError):
            fa.paged_tables(lens, _i32([1, 1]), table, pages, page_size, num_pages, 2)


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^31 elements: slots and pages at its far end."""
    ps, Hkv, d = 256, 8, 128
    pages = (2 ** 31 // (ps * Hkv * d)) + 40
    kc, vc = (torch.zeros(pages, Hkv, ps, d, dtype=BF, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(4)
    n = 300
    k, v = (torch.randn(n, Hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(1, 16, d, generator=g, device="cuda").to(BF)
    near, far = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in ([1, 0], [pages - 1, pages - 2]))
    out = []
    for table in (near, far):
        at = torch.arange(n, device="cuda")
        slots = (table[0, (at // ps)] * ps + at % ps).to(torch.int32)
        fa.paged_append(k, v, slots, kc, vc)
        out.append(fa.attention_fwd_paged(q, kc, vc, table, _i32([n])))
        out.append(fa.attention_fwd_paged_prefix(q, kc, vc, table[0].contiguous(), n - 1, table, _i32([1])))
    assert torch.equal(kc[1, :, :], kc[pages - 1]) and torch.equal(vc[0, :, :44], vc[pages - 2, :, :44])
    assert _lib.fa_get_device_status() == _lib.FA_OK
    assert torch.equal(out[0][0], out[2][0]) and torch.equal(out[0][1], out[2][1])
    assert torch.equal(out[1][0], out[3][0]) and torch.equal(out[1][1], out[3][1])
