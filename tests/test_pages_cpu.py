"""Refusals of the entry points for branching requests, none of which launches
anything, and the references that the GPU tests hold them to."""
import pytest
import torch

from _pages import compact_reference, fork_reference, free_reference

FAKE = 1 << 20  # an aligned non-null value; never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from exact_attention_85_gb300 import _lib, build
    build.build()
    return _lib.load()


def _fork(lib, src=FAKE, dst=2 * FAKE, lens=3 * FAKE, table=4 * FAKE, free=5 * FAKE, start=None, shares=6 * FAKE,
          copies=7 * FAKE, counts=8 * FAKE, F=4, B=8, max_pages=8, page_size=16, num_pages=64, num_free=32):
    return lib.fa_paged_fork(src, dst, lens, table, free, start, shares, copies, counts, F, B, max_pages, page_size,
                             num_pages, num_free, None)


@pytest.mark.parametrize("bad,status", [
    (dict(src=None), 1), (dict(dst=None), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(shares=None), 1),
    (dict(copies=None), 1), (dict(counts=None), 1), (dict(free=None), 1), (dict(F=0), 1), (dict(B=0), 1),
    (dict(F=9), 1), (dict(max_pages=0), 1), (dict(num_free=-1), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
    (dict(src=FAKE + 2), 1), (dict(start=FAKE + 1), 1), (dict(counts=8 * FAKE + 2), 1),
    (dict(lens=FAKE), 1), (dict(start=8 * FAKE), 1), (dict(shares=3 * FAKE), 1), (dict(copies=4 * FAKE), 1),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(F=8193, B=10000), 2),
    (dict(max_pages=1 << 28), 2), (dict(num_pages=1 << 28), 2), (dict(B=16384, max_pages=1 << 17), 2),
])
def test_fork_refuses(lib, bad, status):
    assert _fork(lib, **bad) == status


def _copy(lib, src=FAKE, dst=FAKE, rows=None, kc=FAKE, vc=FAKE, n=4, Hkv=2, d=128, page_size=16, num_pages=64, dtype=1):
    return lib.fa_paged_copy(src, dst, rows, kc, vc, n, Hkv, d, page_size, num_pages, dtype, None)


@pytest.mark.parametrize("bad,status", [
    (dict(src=None), 1), (dict(dst=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(n=0), 1), (dict(Hkv=0), 1),
    (dict(num_pages=0), 1), (dict(dtype=2), 1), (dict(kc=FAKE + 8), 1), (dict(vc=FAKE + 8), 1), (dict(src=FAKE + 2), 1),
    (dict(dst=FAKE + 1), 1), (dict(rows=FAKE + 3), 1), (dict(d=96), 2), (dict(page_size=24), 2),
    (dict(num_pages=1 << 30, Hkv=4), 2), (dict(n=0x7FFFFFFF, page_size=256), 2), (dict(Hkv=1 << 20, page_size=256, num_pages=1), 2),
])
def test_copy_refuses(lib, bad, status):
    assert _copy(lib, **bad) == status


def _compact(lib, keep=FAKE, keep_lens=FAKE, base=FAKE, table=FAKE, kc=FAKE, vc=FAKE, B=4, max_keep=8, max_pages=8,
             Hkv=2, d=128, page_size=16, num_pages=64, dtype=1):
    return lib.fa_paged_compact(keep, keep_lens, base, table, kc, vc, B, max_keep, max_pages, Hkv, d, page_size,
                                num_pages, dtype, None)


@pytest.mark.parametrize("bad,status", [
    (dict(keep=None), 1), (dict(keep_lens=None), 1), (dict(base=None), 1), (dict(table=None), 1), (dict(kc=None), 1),
    (dict(vc=None), 1), (dict(B=0), 1), (dict(max_keep=0), 1), (dict(max_pages=0), 1), (dict(Hkv=0), 1),
    (dict(dtype=-1), 1), (dict(kc=FAKE + 4), 1), (dict(vc=FAKE + 8), 1), (dict(keep=FAKE + 2), 1),
    (dict(base=FAKE + 2), 1), (dict(table=FAKE + 1), 1), (dict(keep_lens=FAKE + 3), 1), (dict(d=32), 2),
    (dict(page_size=8), 2), (dict(B=1 << 27), 2), (dict(max_pages=1 << 28), 2), (dict(B=1 << 16, max_pages=1 << 16), 2),
])
def test_compact_refuses(lib, bad, status):
    assert _compact(lib, **bad) == status


def _free(lib, old=FAKE, new=2 * FAKE, table=3 * FAKE, free=4 * FAKE, start=5 * FAKE, shares=None, counts=6 * FAKE, B=4,
          max_pages=8, page_size=16, num_pages=64, num_free=32):
    return lib.fa_paged_free(old, new, table, free, start, shares, counts, B, max_pages, page_size, num_pages, num_free,
                             None)


@pytest.mark.parametrize("bad,status", [
    (dict(old=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(free=None), 1), (dict(start=None), 1),
    (dict(counts=None), 1), (dict(B=0), 1), (dict(max_pages=0), 1), (dict(num_free=-1), 1), (dict(num_pages=0), 1),
    (dict(old=FAKE + 2), 1), (dict(shares=FAKE + 1), 1), (dict(counts=5 * FAKE), 1), (dict(free=3 * FAKE), 1),
    (dict(shares=4 * FAKE), 1), (dict(shares=6 * FAKE), 1), (dict(page_size=8), 2), (dict(page_size=100), 2),
    (dict(B=16385), 2), (dict(max_pages=1 << 28), 2), (dict(num_pages=1 << 28), 2), (dict(B=16384, max_pages=65537), 2),
])
def test_free_refuses(lib, bad, status):
    assert _free(lib, **bad) == status


def test_fork_reference_by_hand():
    table = [[5, 6, 7], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    lens, t, shares, copies, counts, bad = fork_reference([0, 0, 0], [1, 2, 3], [36, 0, 0, 9], table, [9, 8, 3], 1, [0] * 10, 16)
    assert lens == [36, 36, 36, 0] and t == [[5, 6, 7], [5, 6, 8], [5, 6, 3], [-1, -1, -1]] and not bad
    assert [p for p in range(10) if shares[p]] == [5, 6] and shares[5] == 2
    assert copies == [[7, 7, -1], [8, 3, -1], [4, 4, 0]] and counts == [3, 1]


def test_free_reference_by_hand():
    # page 2 is held twice and given up twice, page 4 held twice and given up once
    free, shares, counts, bad = free_reference([48, 40], [16, 0], [[1, 2, 4], [3, 2, 0]], [9] * 6, 5, [0, 0, 1, 0, 1], 16, 5)
    assert free == [9, 9, 2, 3, 0, 9] and shares == [0, 0, 0, 0, 0] and counts == [2, 0] and not bad


def test_compact_reference_by_hand():
    cache = torch.arange(3 * 16.0).reshape(3, 1, 16, 1)
    out = compact_reference(cache, [[1, 16, 17]], [3], [1], [[2, 0]])
    # tokens 2, 17, 18 of pages 2, 0 become 1, 2, 3
    assert out[2, 0, :5, 0].tolist() == [32, 34, 1, 2, 36] and torch.equal(out[:2], cache[:2])
