"""The paged-cache operators on streams that the caller names."""
import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import Problem, check, tables_reference

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _named(how):
    """(stream to write the inputs on, the same as the call's argument)"""
    if how == "handle of the default stream":
        return torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream
    s = torch.cuda.Stream()
    return s, s if how == "stream" else s.cuda_stream


HOW = ["stream", "handle", "handle of the default stream"]


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("prefix", [0, 100])
def test_forward_runs_in_order_on_the_named_stream(cuda_lib, how, prefix):
    """q is written late on the named stream; the call, made while another
    one is current, has to read it."""
    p = Problem([150, 90, 200], [2, 1, 190], 4, 2, 64, 16, torch.bfloat16, 0, prefix)
    q, late = p.q.cuda(), torch.zeros_like(p.q).cuda()
    args = [late, p.k_cache.cuda(), p.v_cache.cuda()]
    fn = fa.attention_fwd_paged
    if prefix:
        fn = fa.attention_fwd_paged_prefix
        args += [_i32(p.front), prefix]
    args += [p.table.cuda(), _i32(p.lens), p.cu.cuda(), p.max_new]
    torch.cuda.synchronize()
    stream, named = _named(how)
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)  # some 50 ms
        late.copy_(q)
    with torch.cuda.stream(torch.cuda.Stream()):
        o, lse = fn(*args, scale=p.scale, stream=named)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    check(o, lse, p.reference(), p.rows)


@pytest.mark.parametrize("how", HOW)
def test_tables_and_append_run_in_order_on_the_named_stream(cuda_lib, how):
    cached, new, pool, total = [15, 0, 33], [2, 20, 1], [9, 4, 7, 3], 23
    table = torch.tensor([[0, -1, -1], [-1, -1, -1], [5, 6, 8]], dtype=torch.int32)
    want = tables_reference(cached, new, table, pool, 0, 16, total)
    dev, late = table.cuda(), _i32([0, 0, 0])
    args = (_i32(cached), late, dev, _i32(pool), 16, 10, total)
    k = torch.randn(total, 2, 64, device="cuda").to(torch.bfloat16)
    kc, vc = (torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = _i32(new)
    torch.cuda.synchronize()
    stream, named = _named(how)
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)
        late.copy_(n)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = fa.paged_tables(*args, stream=named)
        fa.paged_append(k, -k, got[2], kc, vc, stream=named)
    torch.cuda.synchronize()
    assert _lib.fa_get_device_status() == _lib.FA_OK
    assert torch.equal(dev.cpu(), want[0])
    for g, w in zip(got, want[1:]):
        assert g.tolist() == w
    slots = got[2].long()
    assert torch.equal(kc.transpose(1, 2).reshape(160, 2, 64)[slots], k)
    assert torch.equal(vc.transpose(1, 2).reshape(160, 2, 64)[slots], -k)
