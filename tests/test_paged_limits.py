"""The paged-cache operators at the limits of their sizes."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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
