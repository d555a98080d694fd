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
