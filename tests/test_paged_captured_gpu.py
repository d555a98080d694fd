"""Captured paged calls behind what a user's step has in front of them:
copies, fills, other streams and kernels that start early."""
import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import Problem, check

pytestmark = pytest.mark.gpu

CASES = [([1] * 5, 0), ([1] * 70, 2000), ([40, 300], 0), ([200, 1, 1, 1, 1, 1], 300), ([100] + [1] * 30, 6000)]


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Call:
    """A forward on tensors of its own, and what is to be copied into them."""

    def __init__(self, new, prefix):
        self.ps = [Problem([n + 50 + 31 * (i % 7) for i, n in enumerate(new)], new, 8, 2, 64, 16, torch.bfloat16, 0,
                           prefix, seed=s, extra_cols=30) for s in (1, 2)]
        self.src = [[p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda(), p.table.cuda(), _i32(p.lens), p.cu.cuda(),
                     _i32(p.front or [0])] for p in self.ps]
        self.at = [torch.zeros_like(x) for x in self.src[0]]
        self.now = [x.clone() for x in self.src[0]]
        self.prefix = prefix

    def load(self, i):
        for x, y in zip(self.now, self.src[i]):
            x.copy_(y)

    def copy_in(self):
        for x, y in zip(self.at, self.now):
            x.copy_(y)  # contiguous and of one type: memory copies, not kernels

    def run(self):
        q, kc, vc, table, lens, cu, front = self.at
        if self.prefix:
            return fa.attention_fwd_paged_prefix(q, kc, vc, front, self.prefix, table, lens, cu, self.ps[0].max_new)
        return fa.attention_fwd_paged(q, kc, vc, table, lens, cu, self.ps[0].max_new)


@pytest.mark.parametrize("new,prefix", CASES)
@pytest.mark.parametrize("fork", [False, True])
def test_captured_behind_copies(cuda_lib, new, prefix, fork):
    c = Call(new, prefix)
    c.load(0)
    c.copy_in()
    c.run()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        if fork:  # the copies on the graph's stream, the call on another, its result read back on the first
            c.copy_in()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                o, lse = c.run()
                o.add_(0)
            torch.cuda.current_stream().wait_stream(side)
        else:
            c.copy_in()
            o, lse = c.run()
        out = o.clone(), lse.clone()
    for i in (1, 0, 1):
        c.load(i)
        for x in c.at:
            x.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        check(*out, c.ps[i].reference(), c.ps[i].rows)
    assert _lib.fa_get_device_status() == _lib.FA_OK


def test_two_graphs_at_once(cuda_lib):
    """Two graphs, each with the workspace of its capture, replayed on two
    streams at the same time."""
    calls = [Call(*CASES[1]), Call(*CASES[3])]
    graphs, outs = [], []
    for c in calls:
        c.load(0)
        c.copy_in()
        c.run()
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in calls]
    for i in (1, 0):
        for c in calls:
            c.load(i)
            c.copy_in()
        torch.cuda.synchronize()
        for _ in range(20):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for c, o in zip(calls, outs):
            check(*o, c.ps[i].reference(), c.ps[i].rows)
    assert _lib.fa_get_device_status() == _lib.FA_OK


@pytest.mark.parametrize("new,prefix", CASES)
def test_one_workspace_for_calls_in_a_row(cuda_lib, new, prefix):
    """A caller's own workspace, full of NaN and used by every call: back to
    back on one stream the next call starts early, and must not write what the
    last one still reads."""
    calls = [Call(new, prefix), Call(new, prefix)]
    calls[1].ps.reverse()
    calls[1].src.reverse()
    for c in calls:
        c.load(0)
        c.copy_in()
    p = calls[0].ps[0]
    n = _lib.fa_fwd_paged_workspace_bytes(len(new), p.total, p.max_new, 8, 2, 64, p.table.shape[1], 16, prefix)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(30):
        q, kc, vc, table, lens, cu, front = calls[i % 2].at
        if prefix:
            got.append(fa.attention_fwd_paged_prefix(q, kc, vc, front, prefix, table, lens, cu, p.max_new, workspace=ws))
        else:
            got.append(fa.attention_fwd_paged(q, kc, vc, table, lens, cu, p.max_new, workspace=ws))
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    for k in (0, 1):
        check(*got[k], calls[k].ps[0].reference(), p.rows)
        for o, lse in got[k::2]:
            assert torch.equal(o, got[k][0]) and torch.equal(lse, got[k][1])


@pytest.mark.parametrize("new,prefix", CASES)
def test_tensors_at_sixteen_bytes(cuda_lib, new, prefix):
    """Every tensor at an address that is a multiple of 16 bytes (4 for the
    whole numbers) and of no more."""
    c = Call(new, prefix)
    p = c.ps[0]

    def shifted(x):
        step = 16 // x.element_size() if x.is_floating_point() else 1
        room = torch.empty(x.numel() + step, dtype=x.dtype, device="cuda")
        at = room[step:].view(x.shape)
        at.copy_(x)
        return at

    q, kc, vc, table, lens, cu, front = map(shifted, c.src[0])
    o, lse = shifted(torch.zeros_like(q)), shifted(torch.zeros(8, p.total, device="cuda"))
    n = _lib.fa_fwd_paged_workspace_bytes(len(new), p.total, p.max_new, 8, 2, 64, p.table.shape[1], 16, prefix)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    if prefix:
        _lib.fa_fwd_paged_prefix(q, kc, vc, front, prefix, table, lens, cu, o, lse, p.max_new, p.scale, ws)
    else:
        _lib.fa_fwd_paged(q, kc, vc, table, lens, cu, o, lse, p.max_new, p.scale, ws)
    assert _lib.fa_get_device_status() == _lib.FA_OK
    check(o, lse, p.reference(), p.rows)
