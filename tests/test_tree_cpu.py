"""Refusals of the forward on trees of drafted tokens, none of which launches
anything, and its workspace's size."""
import random

import pytest
import torch

from _tree import TreeProblem, path_of, random_tree

FAKE = 1 << 20  # an aligned non-null value; never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from exact_attention_85_gb300 import _lib, build
    build.build()
    return _lib.load()


def _tree(lib, q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lens=FAKE, cu=FAKE, parents=FAKE, o=FAKE, lse=FAKE, B=4, total=80,
          max_new=20, Hq=4, Hkv=2, d=128, max_pages=64, page_size=16, num_pages=64, window=0, scale=0.1, dtype=1, ws=FAKE,
          ws_bytes=1 << 40):
    return lib.fa_fwd_paged_tree(q, kc, vc, table, lens, cu, parents, o, lse, B, total, max_new, Hq, Hkv, d, max_pages,
                                 page_size, num_pages, window, scale, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(cu=None), 1), (dict(cu=None, max_new=1), 1), (dict(parents=None), 1), (dict(o=None), 1), (dict(lse=None), 1),
    (dict(parents=FAKE + 2), 1), (dict(q=FAKE + 8), 1), (dict(lse=FAKE + 4), 1), (dict(cu=FAKE + 2), 1), (dict(B=0), 1),
    (dict(total=0), 1), (dict(max_new=0), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(window=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(dtype=2), 1), (dict(max_pages=0), 1),
    (dict(max_new=1025), 2), (dict(d=96), 2), (dict(page_size=24), 2), (dict(max_pages=1 << 28), 2),
    (dict(B=(1 << 20) + 1, max_pages=1), 2), (dict(total=1 << 30), 2),
    (dict(ws=None), 3), (dict(ws=FAKE + 16), 3), (dict(ws_bytes=1000), 3),
])
def test_tree_refuses(lib, bad, status):
    assert _tree(lib, **bad) == status


def test_tree_workspace(lib):
    size = lib.fa_fwd_paged_tree_workspace_bytes
    args = (4, 80, 20, 4, 2, 128, 64, 16)
    need = size(*args)
    # behind the chain's
    assert need > lib.fa_fwd_paged_workspace_bytes(*args, 0) > 0
    assert _tree(lib, ws_bytes=need - 1) == 3
    # up to 16 rows a key/value head: the paths are in registers
    few = (4, 32, 8, 4, 2, 128, 64, 16)
    assert size(*few) == lib.fa_fwd_paged_workspace_bytes(*few, 0)
    for i, x in ((0, 0), (1, 0), (2, 0), (2, 1025), (3, 3), (4, 0), (5, 96), (6, 0), (6, 1 << 28), (7, 8)):
        assert size(*args[:i], x, *args[i + 1:]) == 0


def test_reference_by_hand():
    p = TreeProblem([[-1, 0, 0, 2, -1]], [12], 1, 1, 64, 16, torch.float16, window=3)
    assert [path_of(p.trees[0], i) for i in range(5)] == [[0], [1, 0], [2, 0], [3, 2, 0], [4]]
    assert [p.visible(0, i) for i in range(5)] == [[5, 6, 7], [6, 7, 8], [6, 7, 9], [7, 9, 10], [5, 6, 11]]
    p.window = 0
    assert p.visible(0, 3) == list(range(8)) + [9, 10]
    # a chain sees what a causal row does
    r = random.Random(0)
    p = TreeProblem([random_tree(r, 6, "chain")], [9], 1, 1, 64, 16, torch.float16, window=4)
    assert [p.visible(0, i) for i in range(6)] == [list(range(i, i + 4)) for i in range(6)]
