"""Refusals of the paged-cache entry points, none of which launches anything,
and the reference that the GPU tests hold them to."""
import pytest
import torch

from _paged import Problem, tables_reference

FAKE = 1 << 20  # an aligned non-null value; never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from exact_attention_85_gb300 import _lib, build
    build.build()
    return _lib.load()


def _tables(lib, cached=FAKE, new=2 * FAKE, free=3 * FAKE, start=None, table=4 * FAKE, lens=5 * FAKE, cu=6 * FAKE,
            slots=7 * FAKE, counts=8 * FAKE, B=4, max_pages=8, page_size=16, num_pages=64, num_free=32, total=4):
    return lib.fa_paged_tables(cached, new, free, start, table, lens, cu, slots, counts, B, max_pages, page_size,
                               num_pages, num_free, total, None)


@pytest.mark.parametrize("bad,status", [
    (dict(cached=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(cu=None), 1),
    (dict(slots=None), 1), (dict(counts=None), 1), (dict(free=None), 1), (dict(B=0), 1), (dict(max_pages=0), 1),
    (dict(total=0), 1), (dict(num_free=-1), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
    (dict(slots=7 * FAKE + 4), 1),            # 16-byte stores
    (dict(cached=FAKE + 2), 1), (dict(start=FAKE + 1), 1),
    (dict(lens=FAKE), 1),                     # the lengths updated in place
    (dict(start=8 * FAKE), 1),                # the counts updated in place
    (dict(cu=2 * FAKE), 1),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
    (dict(B=16385), 2), (dict(max_pages=1 << 28), 2), (dict(num_pages=1 << 28), 2), (dict(B=16384, max_pages=1 << 17), 2),
])
def test_tables_refuses(lib, bad, status):
    assert _tables(lib, **bad) == status


def _append(lib, k=FAKE, v=FAKE, slots=FAKE, kc=FAKE, vc=FAKE, total=4, Hkv=2, d=128, page_size=16, num_pages=64,
            dtype=1):
    return lib.fa_paged_append(k, v, slots, kc, vc, total, Hkv, d, page_size, num_pages, dtype, None)


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(total=0), 1), (dict(Hkv=0), 1), (dict(num_pages=0), 1), (dict(dtype=2), 1), (dict(k=FAKE + 8), 1),
    (dict(vc=FAKE + 8), 1), (dict(slots=FAKE + 2), 1), (dict(d=96), 2), (dict(page_size=24), 2),
    (dict(num_pages=1 << 30, Hkv=4), 2),
])
def test_append_refuses(lib, bad, status):
    assert _append(lib, **bad) == status


def _paged(lib, q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lens=FAKE, cu=FAKE, o=FAKE, lse=FAKE, B=4, total=8, max_new=2,
           Hq=4, Hkv=2, d=128, max_pages=64, page_size=16, num_pages=64, window=0, scale=0.1, dtype=1, ws=FAKE,
           ws_bytes=1 << 40, front=None, prefix=None):
    rest = (o, lse, B, total, max_new, Hq, Hkv, d, max_pages, page_size, num_pages, window, scale, dtype, ws, ws_bytes,
            None)
    if prefix is None:
        return lib.fa_fwd_paged(q, kc, vc, table, lens, cu, *rest)
    return lib.fa_fwd_paged_prefix(q, kc, vc, front, prefix, table, lens, cu, *rest)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(o=None), 1), (dict(lse=None), 1), (dict(B=0), 1), (dict(total=0), 1), (dict(max_new=0), 1), (dict(Hq=0), 1),
    (dict(Hkv=0), 1), (dict(Hq=5), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1), (dict(window=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(dtype=3), 1),
    (dict(q=FAKE + 8), 1), (dict(kc=FAKE + 8), 1), (dict(o=FAKE + 4), 1), (dict(table=FAKE + 1), 1),
    (dict(lens=FAKE + 2), 1), (dict(cu=FAKE + 3), 1),
    (dict(cu=None), 1),                       # several rows a request need offsets
    (dict(cu=None, max_new=1, total=3), 1),   # fewer rows than requests
    (dict(d=32), 2), (dict(d=256), 2), (dict(page_size=8), 2), (dict(page_size=96), 2), (dict(max_pages=1 << 28), 2),
    (dict(num_pages=1 << 28), 2), (dict(total=1 << 30), 2), (dict(B=1 << 20, max_pages=1 << 12), 2),
    (dict(B=1 << 30, max_pages=1, total=1 << 20), 2), (dict(B=(1 << 20) + 1, max_pages=1), 2), (dict(Hkv=1 << 25, Hq=1 << 25, num_pages=1), 2),
    (dict(ws=None), 3), (dict(ws=FAKE + 16), 3), (dict(ws_bytes=0), 3),
])
@pytest.mark.parametrize("prefix", [None, 100])
def test_forward_refuses(lib, bad, status, prefix):
    assert _paged(lib, **{**bad, "front": FAKE, "prefix": prefix}) == status


def test_prefix_refuses(lib):
    assert _paged(lib, front=None, prefix=100) == 1
    assert _paged(lib, front=FAKE, prefix=0) == 1
    assert _paged(lib, front=FAKE, prefix=-5) == 1
    assert _paged(lib, front=FAKE + 2, prefix=5) == 1
    assert _paged(lib, front=FAKE, prefix=0x7FFFFFFF) == 2


def test_workspace_bytes(lib):
    size = lib.fa_fwd_paged_workspace_bytes
    assert size(4, 8, 2, 4, 2, 128, 64, 16, 0) > 0
    assert size(4, 8, 2, 4, 2, 128, 8, 16, 0) == 0  # no sequence of this table is divided
    for bad in [(0, 8, 2, 4, 2, 128, 8, 16, 0), (4, 0, 2, 4, 2, 128, 8, 16, 0), (4, 8, 0, 4, 2, 128, 8, 16, 0),
                (4, 8, 2, 5, 2, 128, 8, 16, 0), (4, 8, 2, 4, 2, 128, 0, 16, 0), (4, 8, 2, 4, 2, 128, 8, 16, -1)]:
        assert size(*bad) == 0
    # one byte less than asked for is refused
    need = size(4, 8, 2, 4, 2, 128, 64, 16, 0)
    assert _paged(lib, ws_bytes=need - 1) == 3


def test_python_layer_refuses_cpu_tensors(lib):
    import exact_attention_85_gb300 as fa
    p = Problem([5, 9], [1, 1], 4, 2, 64, 16, torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        fa.attention_fwd_paged(p.q, p.k_cache, p.v_cache, p.table, i32(5, 9))
    with pytest.raises(ValueError):
        fa.paged_append(p.q[:, :2], p.q[:, :2], i32(0, 1), p.k_cache, p.v_cache)
    with pytest.raises(ValueError):
        fa.paged_tables(i32(5, 9), i32(1, 1), p.table, i32(3, 4), 16, p.num_pages, 2)


def test_tables_reference_by_hand():
    """Two pages of 16 left for three requests: 10 -> 20 takes one, 0 -> 17
    would take two and is not served, 5 -> 6 needs none."""
    table = torch.full((3, 3), -1, dtype=torch.int32)
    table[0, 0], table[2, 0] = 4, 9
    t, lens, cu, slots, counts = tables_reference([10, 0, 5], [10, 17, 1], table, [7, 2], 0, 16, 30)
    assert t.tolist() == [[4, 7, -1], [-1, -1, -1], [9, -1, -1]]
    assert lens == [20, 0, 6] and cu == [0, 10, 27, 28]
    assert slots == [74, 75, 76, 77, 78, 79, 112, 113, 114, 115] + [-1] * 17 + [149] + [-1, -1]
    assert counts == [1, 1]
