"""The paged-cache operators at the limits of their sizes."""
import os
import subprocess
import sys

import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import Problem, check
from test_paged_gpu import ATTENTION, _run

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BF, HF = torch.bfloat16, torch.float16


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


# ------------------------------------------- shared memory of the tables

# a token each for B requests of one full 16-token page: a new page each
TABLES = r'''
import sys, threading, torch
import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

def data(B):
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(B, **i32)[:, None].repeat(1, 2)
    return torch.full((B,), 16, **i32), torch.ones(B, **i32), table, B + torch.arange(B, **i32), 16, 2 * B, B

def call(args):
    return fa.paged_tables(*args)[2]

def right(B, args, slots):
    want = 16 * (B + torch.arange(B, dtype=torch.int32, device="cuda"))
    assert torch.equal(slots, want) and torch.equal(args[2][:, 1], args[3])
    assert _lib.fa_get_device_status() == _lib.FA_OK
'''


def _fresh_process(program):
    """What a kernel is allowed outlasts a call, so each order of calls needs
    a process of its own."""
    r = subprocess.run([sys.executable, "-c", TABLES + program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.gpu
def test_tables_around_48_kilobytes(cuda_lib):
    """12 B + 4 dynamic bytes and the kernel's static ones pass the 48 KB that
    need no opt-in between B = 4083 and B = 4096; smaller calls come first,
    so that none finds the limit raised by a larger one."""
    _fresh_process(r'''
for B in (2730, 2731, 4083, 4084, 4090, 4095, 4096, 5000):
    args = data(B)
    right(B, args, call(args))
''')


@pytest.mark.gpu
def test_tables_of_two_threads(cuda_lib):
    """Two host threads with tables of different sizes, both past 48 KB: one's
    call must not take the other's shared memory away."""
    _fresh_process(r'''
sizes, errors = (4200, 16384), []
def work(B):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            args = data(B)
            for _ in range(3000):
                slots = call(args)
            torch.cuda.current_stream().synchronize()
            done[B] = args, slots
    except Exception as e:
        errors.append(e)
done = {}
threads = [threading.Thread(target=work, args=(B,)) for B in sizes]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
for B in sizes:
    right(B, *done[B])
''')


# ------------------------------------------------ plan of long requests

PLAN = r'''
#include <cstdio>
#include <cstdlib>
#include "paged_dev.cuh"
// per case: rows, heads per key/value head, own keys, window, prefix
int main(int argc, char **argv) {
    for (int i = 1; i + 4 < argc; i += 5) {
        fa::PagedArgs a{};
        const fa::Request r{0, atoi(argv[i]), atoi(argv[i + 2])};
        const fa::FastDiv group = fa::fast_div(atoi(argv[i + 1]));
        a.window = atoi(argv[i + 3]);
        a.prefix_len = atoi(argv[i + 4]);
        const int nb = fa::blocks_of(r, group);
        long long sum = 0;
        int longest = 0;
        for (int lane = 0; lane < 32; ++lane)  // as the kernel's lanes share them
            sum += a.prefix_len ? fa::blocks_tiles<true>(a, group, r, lane, nb, 32, longest)
                                : fa::blocks_tiles<false>(a, group, r, lane, nb, 32, longest);
        printf("%d %lld %d\n", nb, sum, longest);
    }
}
'''


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from exact_attention_85_gb300 import build
    tmp = tmp_path_factory.mktemp("plan")
    src, exe = tmp / "plan.cu", tmp / "plan"
    src.write_text(PLAN)
    r = subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def run(cases):
        out = subprocess.run([str(exe)] + [str(x) for c in cases for x in c], capture_output=True, text=True, timeout=60)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]

    return run


def _tiles(lo, hi):
    return max(1, -(-hi // 128) - lo // 128)


def _plan_by_hand(rows, group, keys, window, prefix):
    """(blocks, key tiles of all blocks, most of one): blocks of 256 rows, a
    row a (token, head) pair, tiles of 128 keys, the prefix' on their own."""
    blocks, total, longest = -(-rows * group // 256), 0, 0
    for k in range(blocks):
        first, last = 256 * k // group, (min(256 * (k + 1), rows * group) - 1) // group
        p0, p1 = keys - rows + first, keys - rows + last  # places of the first and the last row's token
        tiles = _tiles(max(0, p0 + 1 - window) if window else 0, max(0, p1 + 1))
        low = min(max(0, prefix + p0 + 1 - window), prefix) if window else 0
        if low < prefix:
            tiles += _tiles(low, prefix)
        total, longest = total + tiles, max(longest, tiles)
    return blocks, total, longest


def test_plan_of_ordinary_requests(plan):
    cases = [(rows, group, keys, window, prefix) for rows, group in [(1, 1), (17, 3), (256, 1), (300, 8), (1000, 5)]
             for keys in (0, 1, rows, rows + 129, 5000) for window in (0, 1, 200) for prefix in (0, 1, 700)]
    assert plan(cases) == [_plan_by_hand(*c) for c in cases]


@pytest.mark.parametrize("case,tiles", [
    # a prompt of n tokens: 128 / (256 / group) blocks of each number of tiles 1 .. n / 128
    ((4194304, 8, 4194304, 0, 0), 4 * 32768 * 32769 // 2),
    ((4194304, 16, 4194304, 0, 0), 8 * 32768 * 32769 // 2),  # wraps to few, not to less than none
    ((1048576, 128, 1048576, 0, 0), 64 * 8192 * 8193 // 2),
    # a chunk of 2^20 tokens behind 15 * 2^20: 122881 .. 131072 tiles
    ((1048576, 8, 16777216, 0, 0), 4 * 8192 * (122881 + 131072) // 2),
    # behind a shared prefix of 65536 tiles, which each of the 32768 blocks has
    ((1048576, 8, 1048576, 0, 8388608), 4 * 8192 * 8193 // 2 + 32768 * 65536),
])
def test_tiles_of_a_long_request_pass_32_bits(plan, case, tiles):
    assert tiles > 2 ** 31
    assert plan([case])[0][1] == tiles == _plan_by_hand(*case)[1]


# ------------------------------------------------------- long sums of O


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads,keys,dtype", [
    (1, 304, 1 << 20, HF),            # few rows: a pair for each block, 2^18 keys a warp
    (3, 304, (1 << 20) + 77, HF),
    (1, 304, 1 << 23, BF),
    (200, 152, 1 << 20, HF),          # many rows: a row block for each SM
    (40, 152, (1 << 20) + 128 * 256 + 77, HF),
    (200, 152, 1 << 22, BF),
    (300, 8, 1 << 22, HF),            # blocks cut among SMs
])
@pytest.mark.parametrize("d", [64, 128])
def test_long_sums_keep_small_terms(cuda_lib, rows, heads, keys, dtype, d):
    """K is 0, so every weight is 1 (or as large as the others), and V is one
    step s above 1 (2^-10 or 2^-7): O is the same number, and every partial
    sum of up to 2^15 keys (fp16; 2^17 bf16) is a multiple of s below 2^16
    (2^18), exact in 26 bits.  A sum of 2^25 s keys and more that is an addend
    of the tensor cores' next product loses the s of every term."""
    ps, step = 256, torch.finfo(dtype).eps
    kc = torch.zeros(2, heads, ps, d, dtype=dtype, device="cuda")
    vc = torch.full_like(kc, 1 + step)
    table = (torch.arange(-(-keys // ps), dtype=torch.int32, device="cuda") % 2)[None].contiguous()
    q = torch.randn(rows, heads, d, device="cuda").to(dtype)
    o, lse = fa.attention_fwd_paged(q, kc, vc, table, _i32([keys]), _i32([0, rows]), rows)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    want = torch.log(torch.arange(keys - rows + 1, keys + 1, dtype=torch.float64, device="cuda"))
    assert (lse.double() - want).abs().max() <= 2.0 ** -22 * (1 + want.max()) + 2.0 ** -23
    assert (o == 1 + step).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in ATTENTION if max(c[1]) * c[2] // c[3] > 16 or len(c[0]) > 60])
def test_tables_of_long_sequences(cuda_lib, case):
    """Ordinary lengths in tables so wide that the 256-row kernel is the one
    for long sums."""
    lens, new, Hq, Hkv, d, ps, dtype, window, prefix = case
    cols = (40_000 if dtype == HF else 140_000) // ps
    p = Problem(lens, new, Hq, Hkv, d, ps, dtype, window, prefix, seed=d + ps, extra_cols=cols)
    check(*_run(p), p.reference(), p.rows)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads,window,prefix", [(200, 152, 0, 0), (40, 152, 50_000, 0), (150, 8, 0, 100_000),
                                                      (1, 304, 0, 70_000)])
def test_growing_scores_over_many_tiles(cuda_lib, rows, heads, window, prefix):
    """Scores that rise through the sequence, so that what was summed is
    scaled down again and again, before and after it leaves the tensor
    cores' memory: against 64 bits."""
    ps, d, keys = 256, 64, 150_000
    pages, front = -(-keys // ps), -(-prefix // ps)
    g = torch.Generator(device="cuda").manual_seed(rows)
    # key j is (j / 2000, 0, ..) and q (1, 0, ..) * sqrt(d): score j / 2000 of all keys
    place = torch.arange((pages + front) * ps, device="cuda", dtype=torch.float64)
    at = torch.where(place < front * ps, place, place - front * ps + prefix)
    kc = torch.zeros(pages + front, 1, ps, d, dtype=torch.float16, device="cuda")
    kc[..., 0] = (at / 2000).to(torch.float16).view(-1, 1, ps)
    vc = torch.randn(kc.shape, generator=g, device="cuda").to(torch.float16) + 1
    k1, v1 = kc[:, 0].reshape(-1, d).double(), vc[:, 0].reshape(-1, d).double()
    k1, v1 = (torch.cat([x[:prefix], x[front * ps:front * ps + keys]]) for x in (k1, v1))
    kc, vc = (x.repeat(1, heads, 1, 1) for x in (kc, vc))
    q = torch.zeros(rows, heads, d, device="cuda", dtype=torch.float16)
    q[..., 0] = d ** 0.5
    table = (front + torch.arange(pages, dtype=torch.int32, device="cuda"))[None].contiguous()
    args = (table, _i32([keys]), _i32([0, rows]), rows)
    if prefix:
        pre = torch.arange(front, dtype=torch.int32, device="cuda")
        o, lse = fa.attention_fwd_paged_prefix(q, kc, vc, pre, prefix, *args, window=window or None)
    else:
        o, lse = fa.attention_fwd_paged(q, kc, vc, *args, window=window or None)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    u = 2.0 ** -11
    for r in sorted({0, rows // 2, rows - 1}):
        hi = prefix + keys - rows + r + 1
        lo = max(0, hi - window) if window else 0
        x = k1[lo:hi, 0]
        p = torch.exp(x - x.max())
        want, weight = p @ v1[lo:hi] / p.sum(), p @ v1[lo:hi].abs() / p.sum()
        # weights: scores up to 125 rounded twice in the exponent's argument, P to 16 bits; sums of 2^15 keys
        # at a time lose 2^-26 a term, each fp32 sum after them 2^-24; O is stored
        e = 2.0 ** -22 * (1 + 125 * 1.5) + 2.0 ** -17
        tol = (2 * (e + u) + 2.0 ** -11) * weight + u * want.abs()
        assert ((o[r].double() - want).abs() <= tol).all()
        want_l = x.max() + torch.log(p.sum())
        assert (lse[:, r].double() - want_l).abs().max() <= e + 2.0 ** -22 * (1 + want_l)


@pytest.mark.gpu
@pytest.mark.parametrize("behind", [0, 37])  # the last key tile full, or with keys that no row sees
def test_a_quarter_billion_keys(cuda_lib, behind):
    """A block of 100 rows for each SM, each over 1.8 million key tiles (more
    than a second): warps that have nothing to do meanwhile must not take that
    for a wait that ran out.  The table names 8 pages again and again, K is 0
    and V is 1, so O is 1: each of the 1800 additions of 2^17 keys' sums is
    off by three roundings at most, 3.2e-4 in all, less than half a step of
    bf16 below 1 (2^-9)."""
    rows, heads, d, ps, keys = 100, 152, 64, 256, 230_000_000 // 128 * 128 + behind
    kc = torch.zeros(8, heads, ps, d, dtype=BF, device="cuda")
    vc = torch.ones_like(kc)
    table = (torch.arange(-(-keys // ps), dtype=torch.int32, device="cuda") % 8)[None].contiguous()
    q = torch.randn(rows, heads, d, device="cuda").to(BF)
    o, lse = fa.attention_fwd_paged(q, kc, vc, table, _i32([keys]), _i32([0, rows]), rows)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    want = torch.log(torch.arange(keys - rows + 1, keys + 1, dtype=torch.float64, device="cuda"))
    # the sums are multiples of 128 below 2^28 but for the last tile's, exact in 32 bits
    assert (lse.double() - want).abs().max() <= 2.0 ** -22 * (1 + want.max()) + 2.0 ** -23
    assert (o == 1).all()


# ------------------------------------------------------- small weights


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads", [(1, 304), (4, 304), (200, 152), (300, 4)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_many_small_weights_beside_a_large_one(cuda_lib, rows, heads, dtype, d):
    """Key 0 scores 17.6 above all others (25.4 in log2): their weights, 2^-25
    each, count together.  P is rounded to the type's precision, in fp16 to no
    less than 2^-25 / 2^7 of the largest weight: n 2^-32 of it at most."""
    ps, keys = 256, 1 << 17
    g = torch.Generator(device="cuda").manual_seed(d)
    kc = torch.zeros(keys // ps, 1, ps, d, dtype=dtype, device="cuda")
    kc[0, 0, 0, 0] = 4
    vc = (1 + 0.1 * torch.randn(kc.shape, generator=g, device="cuda")).to(dtype)
    vc[0, 0, 0] = 0
    q = torch.zeros(rows, heads, d, dtype=dtype, device="cuda")
    q[..., 0] = 4.4 * d ** 0.5
    table = torch.arange(keys // ps, dtype=torch.int32, device="cuda")[None].contiguous()
    o, lse = fa.attention_fwd_paged(q, kc.repeat(1, heads, 1, 1), vc.repeat(1, heads, 1, 1), table, _i32([keys]),
                                    _i32([0, rows]), rows)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    k, v = kc.reshape(-1, d).double(), vc.reshape(-1, d).double()
    u = torch.finfo(dtype).eps / 2
    for r in {0, rows - 1}:
        n = keys - rows + r + 1
        x = k[:n] @ q[r, 0].double() / d ** 0.5
        p = torch.exp(x - x.max())
        want = p @ v[:n] / p.sum()
        # dot products of one term; the exponent's argument is rounded twice; sums of 2^15 keys at a time lose 2^-11
        e = 2.0 ** -22 * (1 + 17.6 * 1.5) + u
        tol = (2 * e + 2.0 ** -11) * want + n * 2.0 ** -32 * v.abs().max() + u * want + 2.0 ** -25
        assert ((o[r].double() - want).abs() <= tol).all()
        want_l = x.max() + torch.log(p.sum())
        assert (lse[:, r].double() - want_l).abs().max() <= e + 2.0 ** -22 * (1 + want_l)



@pytest.mark.gpu
@pytest.mark.parametrize("rows,keys", [(1, 700), (4, 5000), (40, 900), (300, 3000)])
@pytest.mark.parametrize("size", [300.0, 3000.0, 8000.0])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_huge_scores_choose_one_key(cuda_lib, rows, keys, size, dtype):
    """Scores up to 2^29, the most that is defined: their fp32 sums are off by
    far more than a unit of the exponent.  O stays finite, and is the value of
    the key that is ahead by more than that error."""
    ps, d, heads = 64, 64, 3
    g = torch.Generator(device="cuda").manual_seed(rows)
    pages = -(-keys // ps)
    kc, vc = (torch.randn(pages, heads, ps, d, generator=g, device="cuda") for _ in range(2))
    kc, vc = kc.mul_(size).clamp_(-6e4, 6e4).to(dtype), vc.to(dtype)
    q = torch.randn(rows, heads, d, generator=g, device="cuda").mul_(size).clamp_(-6e4, 6e4).to(dtype)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].repeat(1, 40).contiguous()
    o, lse = fa.attention_fwd_paged(q, kc, vc, table, _i32([keys]), _i32([0, rows]), rows)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    k, v = (x.transpose(0, 1).reshape(heads, -1, d).double() for x in (kc, vc))
    checked = 0
    for r in range(rows):
        n = keys - rows + r + 1
        x = torch.einsum("hd,hnd->hn", q[r].double(), k[:, :n]) / d ** 0.5
        error = d * 2.0 ** -23 * torch.einsum("hd,hnd->hn", q[r].double().abs(), k[:, :n].abs()).amax(1) / d ** 0.5
        top, at = x.topk(2, 1)
        assert x.abs().max() < 2 ** 29
        for h in range(heads):
            if top[h, 0] - top[h, 1] > 4 * error[h] + 60:
                checked += 1
                assert torch.equal(o[r, h].double(), v[h, at[h, 0]])
                assert (lse[h, r].double() - top[h, 0]).abs() <= error[h] + 2.0 ** -21 * top[h, 0].abs()
    assert checked > rows * heads // 2


# ------------------------------------------------------- workspace


@pytest.mark.parametrize("bad", [dict(d=96), dict(d=32), dict(page_size=8), dict(page_size=24), dict(page_size=512),
                                 dict(B=1 << 20, max_pages=1 << 12), dict(total=1 << 30), dict(prefix_len=-1),
                                 dict(prefix_len=2 ** 31 - 1), dict(Hkv=1 << 25, Hq=1 << 25)])
def test_workspace_of_refused_sizes_is_none(bad):
    """0 bytes for sizes that the forward refuses, whichever rule they break."""
    from exact_attention_85_gb300 import build
    build.build()
    sizes = dict(B=4, total=8, max_new=2, Hq=4, Hkv=2, d=128, max_pages=64, page_size=16, prefix_len=0)
    assert _lib.fa_fwd_paged_workspace_bytes(**sizes) > 0
    assert _lib.fa_fwd_paged_workspace_bytes(**{**sizes, **bad}) == 0


# ------------------------------------------------------- far places


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens", [([2000], [0]), ([2000, 40], [3, 60]), ([1500, 1, 1, 1, 1, 1], [0, 5, 0, 90, 1, 3])])
def test_window_of_two_billion_in_a_wide_table(cuda_lib, new, lens):
    """A window that is almost all of the widest table, and rows that stand
    in the prefix (more rows than keys of their own): place - window is less
    than 32 bits hold.  The window hides nothing, so O is that without one."""
    ps, prefix, Hq, d = 256, 5000, 2, 64
    cols = (2 ** 31 - 1024 - prefix) // ps
    window = cols * ps + prefix - 50
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn(30, 1, ps, d, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(sum(new), Hq, d, generator=g, device="cuda").to(BF)
    table = torch.zeros(len(new), cols, dtype=torch.int32, device="cuda")
    table[:, 0] = 20 + torch.arange(len(new), dtype=torch.int32, device="cuda")
    cu = _i32([sum(new[:b]) for b in range(len(new) + 1)])
    args = (q, kc, vc, _i32(range(20)), prefix, table, _i32(lens), cu, max(new))
    o, lse = fa.attention_fwd_paged_prefix(*args, window=window)
    whole, whole_lse = fa.attention_fwd_paged_prefix(*args)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    assert torch.isfinite(whole_lse).all()
    assert torch.equal(o, whole) and torch.equal(lse, whole_lse)


# ------------------------------------------------------- sizes past 32 bits


def test_rows_past_32_bits_are_refused_before_they_are_allocated():
    i32 = dict(dtype=torch.int32)
    one, table = torch.ones(1, **i32), torch.zeros(1, 4, **i32)
    with pytest.raises(ValueError, match="total"):
        fa.paged_tables(one, one, table, one, 16, 8, 2 ** 32 + 2)


@pytest.mark.gpu
def test_tensors_past_32_bits_are_refused(cuda_lib):
    """Of a table of 2^32 + 2 columns or a free list as long, the low 32 bits
    of the size would be passed on."""
    far = torch.empty(1, 2 ** 32 + 2, dtype=torch.int32, device="cuda")
    one, table = _i32([1]), _i32([0, 0])[None]
    q = torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    kc = torch.zeros(2, 1, 16, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="max_pages"):
        fa.paged_tables(one, one, far, one, 16, 8, 1)
    with pytest.raises(ValueError, match="free_pages"):
        fa.paged_tables(one, one, table, far[0], 16, 8, 1)
    with pytest.raises(ValueError, match="max_pages"):
        fa.attention_fwd_paged(q, kc, kc, far, one)
    with pytest.raises(ValueError, match="max_pages"):
        fa.attention_fwd_paged_prefix(q, kc, kc, one, 16, far, one)


# ------------------------------------------------------- most requests


@pytest.mark.gpu
@pytest.mark.parametrize("rows,long", [(1, 0), (17, 0), (1, 300)])
@pytest.mark.parametrize("prefix", [0, 40])
def test_a_million_requests(cuda_lib, rows, long, prefix):
    """FA_PAGED_MAX_B requests of one row (few-row kernel), of 17 (256-row
    kernel), and of one but for a long one in the middle and at the end
    (both): a sample of them against 64 bits."""
    B, ps, d, pages = 1 << 20, 16, 64, 64
    g = torch.Generator(device="cuda").manual_seed(rows)
    kc, vc = (torch.randn(pages, 1, ps, d, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.randint(pages, (B, 24), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(rows, 49, (B,), generator=g, device="cuda", dtype=torch.int32)
    new = torch.full((B,), rows, dtype=torch.int64, device="cuda")
    for b in (B // 2, B - 1) if long else ():
        new[b], lens[b] = long, 380
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = new.cumsum(0)
    q = torch.randn(int(cu[-1]), 1, d, generator=g, device="cuda").to(BF)
    args = (table, lens, cu, max(rows, long))
    front = _i32(range(-(-prefix // ps)))
    if prefix:
        o, lse = fa.attention_fwd_paged_prefix(q, kc, vc, front, prefix, *args)
    else:
        o, lse = fa.attention_fwd_paged(q, kc, vc, *args)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    k1, v1 = kc[:, 0].double(), vc[:, 0].double()
    for b in [0, 1, 31, 32, 255, 256, 257, 5000, B // 2 - 1, B // 2, B // 2 + 1, B - 2, B - 1]:
        n, m, r0 = int(lens[b]), int(new[b]), int(cu[b])
        ids = table[b].long()
        k, v = (torch.cat([x[front.long()].reshape(-1, d)[:prefix], x[ids].reshape(-1, d)[:n]]) for x in (k1, v1))
        x = q[r0:r0 + m, 0].double() @ k.T / d ** 0.5
        place = prefix + n - m + torch.arange(m, device="cuda")
        x.masked_fill_(torch.arange(prefix + n, device="cuda") > place[:, None], -float("inf"))
        p = torch.softmax(x, 1)
        want, weight = p @ v, p @ v.abs()
        # P and O rounded to bf16 (2^-8 each, P also in the sum); the fp32 errors of scores below 8 are below 2^-17
        tol = (2 * 2.0 ** -8 + 2.0 ** -15) * weight + 2.0 ** -8 * want.abs()
        assert ((o[r0:r0 + m, 0].double() - want).abs() <= tol).all(), b
        assert (lse[0, r0:r0 + m].double() - torch.logsumexp(x, 1)).abs().max() <= 2.0 ** -16, b
