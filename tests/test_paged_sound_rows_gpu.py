"""A request whose values on the device break the rules leaves the rows of
all the others right."""
import pytest
import torch

import exact_attention_85_gb300 as fa
from exact_attention_85_gb300 import _lib

from _paged import Problem, check

pytestmark = pytest.mark.gpu

# requests of one row; of many; of few and many (both kernels); short and long
NEW = [[1] * 6, [30, 70, 40, 1, 90, 33], [2, 1, 190, 3, 1, 1, 1, 2], [1, 60, 1, 1, 300, 1, 1, 1]]


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("prefix", [0, 40, 6000])
@pytest.mark.parametrize("where", ["first", "middle", "longest", "last"])
@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "rows"])
def test_sound_requests_beside_an_unsound_one(cuda_lib, what, where, prefix, new):
    p = Problem([150 + 41 * i % 97 + n for i, n in enumerate(new)], new, 4, 2, 64, 16, torch.bfloat16, 0, prefix,
                extra_cols=60)
    bad = {"first": 0, "middle": len(new) // 2, "longest": new.index(max(new)), "last": len(new) - 1}[where]
    lens, table, most = list(p.lens), p.table.clone(), p.max_new
    unsound = {bad}
    if what == "page":
        table[bad, 1] = p.num_pages
    elif what == "negative page":
        table[bad, 0] = -2 ** 31
    elif what == "length":
        lens[bad] = p.table.shape[1] * 16 + 1
    elif what == "negative length":
        lens[bad] = -1
    else:
        # a bound that some requests do not keep
        if max(new) == 1:
            pytest.skip("one row is the least bound")
        most = max(n for n in new if n < max(new))
        unsound = {b for b, n in enumerate(new) if n > most}
    args = (p.q.cuda(), p.k_cache.cuda(), p.v_cache.cuda())
    tail = (table.cuda(), _i32(lens), p.cu.cuda(), most)
    if prefix:
        o, lse = fa.attention_fwd_paged_prefix(*args, _i32(p.front), prefix, *tail, scale=p.scale)
    else:
        o, lse = fa.attention_fwd_paged(*args, *tail, scale=p.scale)
    assert _lib.fa_get_device_status() == _lib.FA_ERR_INVALID_ARG
    want = p.reference()
    for b, n in enumerate(new):
        if b in unsound:
            continue
        lo, hi = int(p.cu[b]), int(p.cu[b + 1])
        check(o[lo:hi], lse[:, lo:hi], (want[0][lo:hi], want[1][:, lo:hi], want[2][lo:hi], want[3][:, lo:hi]), hi - lo)
    assert _lib.fa_get_device_status() == _lib.FA_OK
