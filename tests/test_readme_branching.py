"""The documents' example of branching requests, run as it stands: the pool's
pages are then held as the counts say or in the list, never both, and every
row's pages hold its own tokens."""
import os
import random
import re

import pytest
import torch

from _pages import compact_reference, copy_reference, fork_reference, free_reference
from _paged import pages_of, tables_reference

PS, PAGES, WIDTH, HKV, D = 64, 30, 6, 2, 64
BASE, DRAFTS = [100, 64], [70, 130]  # rejected drafts end pages of their own, and begin the last kept one


def example():
    """The block of README.md that calls the operators of branching requests."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    found = [b for b in blocks if "paged_fork(" in b]
    assert len(found) == 1
    return found[0]


class Reference:
    """The public functions by the tests' references, in place like the kernels."""

    @staticmethod
    def attention_fwd_paged_tree(*args):
        return None, None

    @staticmethod
    def paged_compact(keep, keep_lens, base_lens, table, *caches):
        for c in caches:
            c.copy_(compact_reference(c, keep.tolist(), keep_lens.tolist(), base_lens.tolist(), table.tolist()))

    @staticmethod
    def paged_copy(src, dst, *caches, rows):
        for c in caches:
            c.copy_(copy_reference(c, src.tolist(), dst.tolist(), rows.tolist()))

    @staticmethod
    def paged_free(old, new, table, free, start, page_size, num_pages, shares=None):
        f, s, counts, unsound = free_reference(old.tolist(), new.tolist(), table.tolist(), free.tolist(), int(start),
                                               shares.tolist(), page_size, num_pages)
        assert not unsound
        free.copy_(torch.tensor(f))
        shares.copy_(torch.tensor(s))
        return torch.tensor(counts, dtype=torch.int32)

    @staticmethod
    def paged_fork(src, dst, lens, table, free, shares, page_size, free_start):
        n, t, s, copies, counts, unsound = fork_reference(src.tolist(), dst.tolist(), lens.tolist(), table.tolist(),
                                                          free.tolist(), int(free_start), shares.tolist(), page_size)
        assert not unsound and not counts[1]
        for x, y in ((lens, n), (table, t), (shares, s)):
            x.copy_(torch.tensor(y))
        return torch.tensor(copies, dtype=torch.int32), torch.tensor(counts, dtype=torch.int32)


def run(fa, device):
    r, g = random.Random(2), torch.Generator().manual_seed(2)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=device)

    # rows 0 and 1 hold their contexts and drafts, rows 2 and 3 nothing
    lens = [b + n for b, n in zip(BASE, DRAFTS)] + [0, 0]
    free = r.sample(range(PAGES), PAGES)
    table, after, cu, _, counts = tables_reference([0] * 4, lens, torch.full((4, WIDTH), -1), free, 0, PS, sum(lens))
    assert after == lens and counts == [sum(pages_of(n, PS) for n in lens), 0]
    caches = [torch.randint(-100, 100, (PAGES, HKV, PS, D), generator=g).to(device, torch.bfloat16) for _ in range(2)]

    def tokens(c, row, n):
        return torch.stack([c[row[t // PS], :, t % PS] for t in range(n)])

    path = [sorted(r.sample(range(n), k)) for n, k in zip(DRAFTS, (7, 5))] + [[], []]
    kept = [len(p) for p in path]
    want = [[torch.cat([x[:b], x[[b + j for j in p]]]) for b, p, x in
             ((BASE[i], path[i], tokens(c, table[i].tolist(), lens[i])) for i in (0, 1))] for c in caches]
    q = torch.randn(sum(DRAFTS), 2 * HKV, D, generator=g).to(device, torch.bfloat16)
    names = dict(
        fa=fa, q=q, k_cache=caches[0], v_cache=caches[1], block_table=table.to(device, torch.int32), lens=i32(lens),
        cu=i32([0, DRAFTS[0], sum(DRAFTS), sum(DRAFTS), sum(DRAFTS)]), max_new=max(DRAFTS),
        parents=i32([r.randint(-1, i - 1) for n in DRAFTS for i in range(n)]),
        path=i32([p + [0] * (max(kept) - len(p)) for p in path]), path_lens=i32(kept), base_lens=i32(BASE + [0, 0]),
        free_pages=i32(free), counts=i32(counts), pages=PAGES, shares=i32([0] * PAGES), src=i32([0, 1]), dst=i32([2, 3]))
    exec(example(), names)
    lens, table = names["lens"].tolist(), names["block_table"].tolist()
    assert lens == 2 * [b + k for b, k in zip(BASE, kept[:2])]
    held = [table[b][c] for b in range(4) for c in range(pages_of(lens[b], PS))]
    shares, start = names["shares"].tolist(), int(names["counts"][0])
    assert int(names["counts"][1]) == 0
    assert sorted(names["free_pages"].tolist()[start:] + list(set(held))) == list(range(PAGES))
    assert [shares[p] for p in range(PAGES)] == [max(0, held.count(p) - 1) for p in range(PAGES)]
    for c, rows in zip(caches, want):
        for b in range(4):
            assert torch.equal(tokens(c, table[b], lens[b]), rows[b % 2])


def test_example_by_references():
    run(Reference, "cpu")


@pytest.mark.gpu
def test_example(cuda_lib):
    import exact_attention_85_gb300 as fa
    run(fa, "cuda")
    torch.cuda.synchronize()
    from exact_attention_85_gb300 import _lib
    assert _lib.fa_get_device_status() == _lib.FA_OK
