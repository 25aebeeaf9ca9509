"""Depths and masks of drafted trees against walks up their parents."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.gpu_util import require_gpu
from tests.tree_util import chains, depths, random_parents, sees, words_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


JUNK = 0x5A5A5A5


def prepared(ns, parents, lead=0, tail=0, max_n=None):
    """(tree, start, error) of requests of ns rows; parents of all T rows."""
    start = np.concatenate([[lead], lead + np.cumsum(ns)]).astype(np.int32)
    T, B = lead + sum(ns) + tail, len(ns)
    flat = np.full(T, JUNK, dtype=np.int32)
    for b, p in enumerate(parents):
        flat[start[b]:start[b + 1]] = p
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    batch = moe.KvBatch(i32(start), i32([0] * B), i32(np.zeros((B, 1))), T, max(ns + [1]) if max_n is None else max_n)
    t = moe.Tree(batch, i32(flat))
    for x in (t.depth, t.above, t.below):
        x.fill_(JUNK)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_tree_prepare(batch, t, err=err)
    return t, start, int(err.item())


def check(t, start, parents):
    depth, above, below = (x.cpu().numpy() for x in (t.depth, t.above, t.below))
    mine = np.zeros(t.T, dtype=bool)
    for b, p in enumerate(parents):
        rows = slice(start[b], start[b + 1])
        mine[rows] = True
        if len(p):
            m = sees(p)
            assert depth[rows].tolist() == depths(p)
            assert (above[rows] == words_of(m, t.words)).all()
            assert (below[rows] == words_of(m.T, t.words)).all()
    for x in (depth, above, below):
        assert (x[~mine] == JUNK).all()


@pytest.mark.parametrize("n", [1, 2, 3, 31, 32, 33, 63, 64, 65, 128, 200, 255, 256])
@pytest.mark.parametrize("spread", [1, 4, 300])
def test_one_tree(n, spread):
    p = random_parents(n, spread, n + spread)
    t, start, err = prepared([n], [p])
    assert err == 0
    check(t, start, [p])


def test_many_trees_beside_rows_of_none():
    r = np.random.RandomState(0)
    ns = [0, 1, 17, 0, 256, 64, 33, 0] + r.randint(0, 100, 300).tolist()
    ps = [random_parents(n, int(r.choice([1, 2, 5, 50])), i) if n else [] for i, n in enumerate(ns)]
    t, start, err = prepared(ns, ps, lead=5, tail=7)
    assert err == 0
    check(t, start, ps)


def test_forests():
    p = [-1, -1, 0, 1, 1, -1, 5, 4]
    t, start, err = prepared([8], [p], max_n=100)
    assert err == 0 and t.words == 4
    check(t, start, [p])


@pytest.mark.parametrize("bad", [0, 3, 2, 100, -2, -2 ** 31, 2 ** 31 - 1])
def test_a_parent_that_is_none_becomes_a_root(bad):
    p = [-1, 0, bad, 2, 1]
    ok = p if 0 <= bad < 2 else [-1, 0, -1, 2, 1]
    t, start, err = prepared([1, 5], [[-1], p])
    assert err == (moe.MOE_OK if ok == p else moe.MOE_ERANGE)
    check(t, start, [[-1], ok])


def test_nodes_past_the_masks():
    p = random_parents(70, 3, 1)
    t, start, err = prepared([70, 5], [p, [-1, 0, 0, 1, 3]], max_n=64)
    assert err == moe.MOE_ERANGE and t.words == 2
    depth, above, below = (x.cpu().numpy() for x in (t.depth, t.above, t.below))
    m = sees(p[:64])
    assert (above[:64] == words_of(m, 2)).all() and (below[:64] == words_of(m.T, 2)).all()
    assert depth[:64].tolist() == depths(p[:64])
    for x in (depth, above, below):
        assert (x[64:70] == 0).all()
    assert depth[70:].tolist() == [0, 1, 1, 2, 3] and (above[70:] == words_of(sees([-1, 0, 0, 1, 3]), 2)).all()


def test_starts_that_decrease_are_reported():
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = moe.KvBatch(i32([0, 3, 1, 4]), i32([0] * 3), i32([[0]] * 3), 4, 3)
    t = moe.Tree(batch, i32([-1, 0, 1, 0]))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_tree_prepare(batch, t, err=err)
    assert err.item() == moe.MOE_ERANGE


def test_chains_agree_with_themselves():
    assert [len(c) for c in chains([-1, 0, 1, 1])] == [1, 2, 3, 3]
